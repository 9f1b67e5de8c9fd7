"""dQ and dK of rows with few allowed keys, whose Delta comes from the weights and not from the
rounded O: within the bounds that leave Delta's error out (oracle/operators.py, exact_delta),
wherever such rows stand and however long the list is that their item walks."""

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
import oracle
from oracle import operators as R
from workloads import configs as W

pytestmark = pytest.mark.gpu

FEW = 127  # keys of a row up to which its Delta is exact


def _tokens(n, heads=2, head_dim=64, kv_heads=0, batch=1):
    """n tokens in 64-slot blocks, every block pair listed: lists of n / 16 pages."""
    nb = -(-n // 64)
    group = (np.arange(n) // 64).astype(np.int32)
    return W.Problem(f"few{n}", batch, heads, head_dim, group, group.copy(), nb, nb,
                     np.arange(0, heads * nb * nb + 1, nb, dtype=np.int64), np.tile(np.arange(nb, dtype=np.int32), heads * nb),
                     900 + n, kv_heads=kv_heads)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _check(p, arrays, cap=0.0, slopes=None, plan=None):
    """Runs both passes; every row with at most FEW keys has an exact Delta in the bounds. Returns their count."""
    t = W.make_tensors(p)
    dev = {k: v.cuda() for k, v in t.items()}
    plan = plan or sp.Plan.from_problem(p)
    sc = sp.Score(softcap=cap, slopes=None if slopes is None else torch.tensor(slopes).float().cuda(),
                  **{k: _i32(v) for k, v in arrays.items()})
    o, lse = sp.spattn_fwd_scored(dev["q"], dev["k"], dev["v"], plan, sc)
    out = dict(zip(("dq", "dk", "dv"), sp.spattn_bwd_scored(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], plan, sc)))
    sp.spattn_check(plan)
    group, few = p.heads // p.n_kv_heads, 0
    for b in range(p.batch):
        pick = lambda n: None if n not in arrays else (arrays[n][b] if np.ndim(arrays[n]) == 2 else arrays[n])  # noqa: E731
        acc = {}
        for h in range(p.heads):
            hk = h // group
            A = oracle.allowed_groups(p.row_ptr, p.kv_groups, p.n_q_groups, p.n_kv_groups, p.graph_head(b, h))
            M = R.score_mask(oracle.token_mask(p.q_group, p.kv_group, A), pick("k_pos"), pick("q_last"), pick("q_doc"),
                             pick("k_doc"))
            f64 = lambda n, i, g: np.where((g >= 0)[:, None], t[n][b, i].double().numpy(), 0.0)  # noqa: E731
            q, do = f64("q", h, p.q_group), f64("do", h, p.q_group)
            k, v = f64("k", hk, p.kv_group), f64("v", hk, p.kv_group)
            z, f = R.scores(q, k, p.scale, cap, 0.0 if slopes is None else float(np.float32(slopes[h])), pick("q_pos"),
                            pick("k_pos"))
            exact = M.sum(axis=1) <= FEW
            few += int((exact & M.any(axis=1)).sum())
            g = R.backward(q, k, v, do, M, z, f, p.scale, exact)
            got = out["dq"][b, h].cpu().double().numpy()
            bad = np.abs(got - g["dq"][0]) > g["dq"][1]
            assert not bad.any(), ("dq", b, h, int(bad.sum()), np.flatnonzero(bad.any(axis=1))[:9])
            assert np.isfinite(got).all()
            for n in ("dk", "dv"):
                val, tol = acc.setdefault((n, hk), [0.0, 0.0])
                acc[(n, hk)] = [val + g[n][0], tol + g[n][1]]
        for (n, hk), (val, tol) in acc.items():
            got = out[n][b, hk].cpu().double().numpy()
            bad = np.abs(got - val) > tol
            assert not bad.any(), (n, b, hk, int(bad.sum()))
    return few


def _docs(n, longest, seed):
    rng = np.random.default_rng(seed)
    return np.repeat(np.arange(n), rng.integers(1, longest + 1, n))[:n]


@pytest.mark.parametrize("pack", ["", "route64", "split", "slot"])
@pytest.mark.parametrize("head_dim,kv_heads", [(64, 2), (128, 1)])
@pytest.mark.parametrize("cap,longest", [(0.0, 3), (15.0, 40), (0.0, 40)])
def test_short_documents_in_long_lists(cap, longest, head_dim, kv_heads, pack, monkeypatch):
    if pack:
        monkeypatch.setenv("SPATTN_PLAN_PACK", pack)
    n = 700  # 44 pages a list
    doc = _docs(n, longest, 3)
    assert _check(_tokens(n, 2, head_dim, kv_heads), dict(q_doc=doc, k_doc=doc), cap) == 2 * n


@pytest.mark.parametrize("n", [40, 300, 1000])
@pytest.mark.parametrize("slopes", [None, [0.05, -0.01]])
def test_causal_documents(n, slopes):
    """The first tokens of every document have 1, 2, 3, .. keys."""
    doc, i = _docs(n, 400, n), np.arange(n)
    arrays = dict(q_doc=doc, k_doc=doc, q_last=i, k_pos=i, q_pos=i)
    assert _check(_tokens(n), arrays, 0.0 if slopes else 8.0, slopes) >= 2 * min(n, 127)


def test_keys_at_the_far_end_of_a_list():
    """Every query attends a few of the last keys, or of the first, alone."""
    n = 900
    i = np.arange(n)
    doc = np.where(i % 2 == 0, 1, 2)
    k_doc = np.full(n, 3)
    k_doc[-5:], k_doc[:128] = 1, 2  # 5 keys for the even queries, 128 for the odd ones
    assert _check(_tokens(n), dict(q_doc=doc, k_doc=k_doc)) == n
    k_doc[127] = 3
    assert _check(_tokens(n), dict(q_doc=doc, k_doc=k_doc)) == 2 * n


@pytest.mark.parametrize("name", ["tiny_onekey", "tiny_svg2", "tiny_gqa", "tiny_empty", "tiny_hedge"])
def test_few_keys_by_the_graph_and_the_masks(name):
    p = W.make_problem(name)
    rng = np.random.default_rng(2)
    _check(p, {}, 10.0)
    arrays = dict(q_doc=rng.integers(-1, 40, p.q_slots), k_doc=rng.integers(-1, 40, p.kv_slots))
    assert _check(p, arrays, 0.0) > 0


def test_documents_in_no_order():
    """Every row's keys are spread over its whole list."""
    n = 1300  # 82 pages a list
    rng = np.random.default_rng(6)
    arrays = dict(q_doc=rng.integers(-1, 12, n), k_doc=rng.integers(-1, 12, n), q_last=rng.integers(0, n, n), k_pos=rng.permutation(n))
    assert n < _check(_tokens(n, 2, 128, 1), arrays, 6.0) <= 2 * n


def test_batches_and_a_device_replan():
    n = 500
    p = _tokens(n, 2, 64, 1, batch=2)
    arrays = {k: np.stack([_docs(n, 5, 1), _docs(n, 60, 2)]) for k in ("q_doc", "k_doc")}
    plan = sp.Plan.from_problem(p)
    assert _check(p, arrays, 0.0, None, plan) > n
    plan.set_graph_device(torch.from_numpy(p.row_ptr).cuda(), torch.from_numpy(p.kv_groups).cuda())
    assert _check(p, arrays, 0.0, None, plan) > n


def test_extreme_caps_and_scores():
    n = 200
    doc = _docs(n, 6, 8)
    for cap in (1e-20, 1e-3, 1e30):
        _check(_tokens(n), dict(q_doc=doc, k_doc=doc), cap)


def test_profiled_calls_give_the_same_bits():
    """(events between the launches keep them from running side by side)"""
    n = 400
    p = _tokens(n)
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    doc = _i32(_docs(n, 9, 4))
    plan, sc = sp.Plan.from_problem(p), sp.Score(q_doc=doc, k_doc=doc)
    o, lse = sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc)
    runs = []
    for on in (False, True, False):
        plan.profile(on)
        runs.append(sp.spattn_bwd_scored(t["q"], t["k"], t["v"], o, lse, t["do"], plan, sc))
    plan.profile(False)
    for r in runs[1:]:
        for x, y in zip(r, runs[0]):
            assert torch.equal(x, y)
    sp.spattn_check(plan)


def _backward_of(p, t, plan, sc):
    o, lse = sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc)
    return (o, lse) + tuple(sp.spattn_bwd_scored(t["q"], t["k"], t["v"], o, lse, t["do"], plan, sc))


def test_replays_with_other_documents():
    """A captured pass lists its rows of few keys anew: documents that change between replays, none among them."""
    n = 700
    p = _tokens(n, 3, 128, 1)
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    doc = _i32(_docs(n, 30, 1))
    plan, sc = sp.Plan.from_problem(p), sp.Score(q_doc=doc, k_doc=doc)
    _backward_of(p, t, plan, sc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = _backward_of(p, t, plan, sc)
    for other in (_docs(n, 200, 2), np.zeros(n), _docs(n, 3, 3), np.full(n, -1), _docs(n, 60, 4)):
        doc.copy_(_i32(other))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        for x, y in zip(got, _backward_of(p, t, plan, sc)):
            assert torch.equal(x, y)
    sp.spattn_check(plan)


def test_two_plans_on_two_streams():
    work = []
    for n, longest in ((900, 40), (640, 7)):
        p = _tokens(n, 4, 64, 2)
        t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
        doc = _i32(_docs(n, longest, n))
        work.append((p, t, sp.Plan.from_problem(p), sp.Score(softcap=9.0, q_doc=doc, k_doc=doc)))
    want = [_backward_of(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = []
    for _ in range(20):
        for w, st in zip(work, streams):
            with torch.cuda.stream(st):
                got.append((w, _backward_of(*w)))
    torch.cuda.synchronize()
    for i, (_, r) in enumerate(got):
        for x, y in zip(r, want[i % 2]):
            assert torch.equal(x, y)
    for w in work:
        sp.spattn_check(w[2])


def test_more_items_than_are_ordered():
    """Lists without an order (their number is above the limit for one): each item is looked at by both passes."""
    n, heads, batch = 320, 20, 80  # 4800 items of 20 pages
    p = _tokens(n, heads, 64, 20, batch=batch)
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = {k: torch.randn((batch, heads, n, 64), generator=gen, device="cuda").bfloat16() for k in ("q", "k", "v", "do")}
    doc = _i32(_docs(n, 20, 5))
    plan = sp.Plan.from_problem(p)
    assert plan.stats()["n_work_fwd"] == 4800
    got = _backward_of(p, t, plan, sp.Score(q_doc=doc, k_doc=doc))
    one = sp.Plan.from_problem(_tokens(n, heads, 64, 20))
    for b in (0, 41, 79):
        alone = _backward_of(p, {k: v[b:b + 1].contiguous() for k, v in t.items()}, one, sp.Score(q_doc=doc, k_doc=doc))
        for x, y in zip(got, alone):
            assert torch.equal(x[b:b + 1], y)
    sp.spattn_check(plan)
