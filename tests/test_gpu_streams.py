"""Calls on an explicit stream: the tensors that a call makes itself (results and
workspaces) come from the pool of that stream, so that no kernel of the
current stream still uses their memory."""

import contextlib

import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
from workloads import configs as W

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def _recorded():
    """The streams on which torch.empty, empty_like and Tensor.new_empty are called, in order."""
    seen = []
    kept = torch.empty, torch.empty_like, torch.Tensor.new_empty

    def wrap(f):
        def g(*a, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return f(*a, **kw)
        return g

    torch.empty, torch.empty_like, torch.Tensor.new_empty = map(wrap, kept)
    try:
        yield seen
    finally:
        torch.empty, torch.empty_like, torch.Tensor.new_empty = kept


def _calls():
    """name -> (tensors that the call makes, call(stream))."""
    p = W.make_problem("tiny_d128")
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    plan = sp.Plan.from_problem(p)
    last = torch.arange(p.q_slots, dtype=torch.int32).cuda()
    sc = sp.Score(softcap=20.0, q_last=last, k_pos=torch.arange(p.kv_slots, dtype=torch.int32).cuda())
    o, lse = sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc)
    o1, lse1 = sp.spattn_fwd(t["q"], t["k"], t["v"], plan)
    q8, qd = sp.quantize_fp8(t["q"])
    k8, kd = sp.quantize_fp8(t["k"])
    freqs, _ = sp.rope_freqs(64)
    paged = sp.PagedPlan(heads=16, kv_heads=2, head_dim=128, page_slots=16, max_seqs=1, max_q=1, max_kv=8000)
    gen = torch.Generator().manual_seed(5)
    cache = [torch.randn((500, 16, 2, 128), generator=gen).bfloat16().cuda() for _ in range(2)]
    table = torch.randperm(500, generator=gen).int()[None].cuda()
    qs, n = torch.tensor([0, 1], dtype=torch.int32).cuda(), torch.tensor([7990], dtype=torch.int32).cuda()
    qp = torch.randn((1, 16, 128), generator=gen).bfloat16().cuda()
    assert paged.workspace_bytes(1) > 0
    torch.cuda.synchronize()
    keep = (plan, paged)
    return keep, {
        "fwd": (2, lambda s: sp.spattn_fwd(t["q"], t["k"], t["v"], plan, stream=s)),
        "bwd": (3, lambda s: sp.spattn_bwd(t["q"], t["k"], t["v"], o1, lse1, t["do"], plan, stream=s)),
        "quantize": (2, lambda s: sp.quantize_fp8(t["q"], stream=s)),
        "fp8": (2, lambda s: sp.spattn_fwd_fp8(q8, k8, qd, kd, t["v"], plan, stream=s)),
        "fwd_scored": (2, lambda s: sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc, stream=s)),
        "bwd_scored": (3, lambda s: sp.spattn_bwd_scored(t["q"], t["k"], t["v"], o, lse, t["do"], plan, sc, stream=s)),
        "rope": (2, lambda s: sp.rope(t["q"], t["k"], last, freqs, stream=s)),
        "paged": (3, lambda s: sp.spattn_paged_fwd(qp, *cache, table, qs, n, paged, stream=s)),
    }


def test_tensors_of_a_call_come_from_its_own_stream():
    keep, calls = _calls()
    side = torch.cuda.Stream()
    raw = torch.cuda.ExternalStream(side.cuda_stream)
    here = torch.cuda.current_stream()
    for name, (count, call) in calls.items():
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        for stream in (side, raw):
            with _recorded() as seen:
                got = call(stream)
            assert seen == [side.cuda_stream] * count, name
            assert torch.cuda.current_stream() == here
            torch.cuda.synchronize()
            for x, y in zip(want, got):
                assert torch.equal(x, y), name
        for stream in (None, here):
            with _recorded() as seen:
                call(stream)
            assert seen == [here.cuda_stream] * count, name
        torch.cuda.synchronize()


def test_paged_calls_on_the_current_and_a_side_stream_at_once():
    """A call of many partial rows in flight on the current stream, its workspace already handed back, and the same
    call on a side stream right behind it: neither may write over the other's partial rows."""
    paged = sp.PagedPlan(heads=16, kv_heads=4, head_dim=128, page_slots=64, max_seqs=1, max_q=96, max_kv=40000)
    gen = torch.Generator().manual_seed(9)
    cache = [torch.randn((625, 64, 4, 128), generator=gen).bfloat16().cuda() for _ in range(2)]
    table = torch.randperm(625, generator=gen).int()[None].cuda()
    lens = [torch.tensor([n], dtype=torch.int32).cuda() for n in (40000, 37777)]
    start = torch.tensor([0, 96], dtype=torch.int32).cuda()
    q = [torch.randn((96, 16, 128), generator=gen).bfloat16().cuda() for _ in range(2)]
    assert paged.workspace_bytes(1) > 0
    want = [sp.spattn_paged_fwd(q[i], *cache, table, start, lens[i], paged) for i in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(15):
        got.append((0, sp.spattn_paged_fwd(q[0], *cache, table, start, lens[0], paged)))
        got.append((1, sp.spattn_paged_fwd(q[1], *cache, table, start, lens[1], paged, stream=side)))
    torch.cuda.synchronize()
    for i, (o, lse) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    sp.spattn_paged_check(paged)
    assert bool(torch.isfinite(want[0][1]).all())


def test_a_forked_stream_inside_a_capture():
    keep, calls = _calls()
    side = torch.cuda.Stream()
    for name in ("fwd_scored", "rope", "paged"):
        call = calls[name][1]
        want = [x.clone() for x in call(None)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            got = call(side)
            here.wait_stream(side)
        for _ in range(3):
            for x in got:
                x.zero_()
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(want, got):
                assert torch.equal(x, y), name
        del g, got
