"""A NaN score in a row that attends something shows: O and LSE of that row are NaN (they
are not those of an empty row), gradients too, and other rows keep their results."""

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
from oracle import operators as R
from workloads import configs as W

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _problem(n, heads=2, head_dim=64):
    """n tokens in 64-slot blocks, each of which attends itself and the one before."""
    nb = -(-n // 64)
    group = (np.arange(n) // 64).astype(np.int32)
    lists = [[a] if a == 0 else [a - 1, a] for a in range(nb)] * heads
    return W.Problem(f"band{n}", 1, heads, head_dim, group, group.copy(), nb, nb,
                     np.cumsum([0] + [len(x) for x in lists]).astype(np.int64), np.concatenate(lists).astype(np.int32), 77)


def _score(n, kind, cap):
    pos = torch.arange(n, dtype=torch.int32).cuda()
    if kind == "none":
        return sp.Score(softcap=cap)
    if kind == "causal":
        return sp.Score(softcap=cap, q_last=pos, k_pos=pos)
    return sp.Score(softcap=cap, slopes=torch.tensor([0.1, 0.01]).cuda(), q_pos=pos, k_pos=pos)


def _mask(p, kind):
    g = p.q_group.astype(np.int64)
    m = (g[:, None] - g[None, :] >= 0) & (g[:, None] - g[None, :] <= 1)
    i = np.arange(len(g))
    return m & (i[None, :] <= i[:, None]) if kind == "causal" else m


@pytest.mark.parametrize("pack", ["", "route64"])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("kind,cap", [("plain", 0.0), ("none", 20.0), ("causal", 0.0), ("causal", 5.0), ("bias", 0.0)])
def test_rows_of_the_plan(kind, cap, head_dim, pack, monkeypatch):
    if pack:
        monkeypatch.setenv("SPATTN_PLAN_PACK", pack)
    n = 300
    p = _problem(n, head_dim=head_dim)
    plan = sp.Plan.from_problem(p)
    sc = None if kind == "plain" else _score(n, kind, cap)
    slopes = [0.1, 0.01] if kind == "bias" else [0.0, 0.0]
    mask = _mask(p, kind)

    def forward(t):
        a = (t["q"], t["k"], t["v"], plan)
        return sp.spattn_fwd(*a) if sc is None else sp.spattn_fwd_scored(*a, sc)

    def backward(t, o, lse):
        a = (t["q"], t["k"], t["v"], o, lse, t["do"], plan)
        return sp.spattn_bwd(*a) if sc is None else sp.spattn_bwd_scored(*a, sc)

    base = W.make_tensors(p)
    i = np.arange(n)
    for name, at in (("q", 70), ("k", 130)):
        t = {k: v.clone().cuda() for k, v in base.items()}
        t[name][0, 1, at, 3] = NAN
        o, lse = forward(t)
        hit = i == at if name == "q" else mask[:, at]
        assert hit.any() and not hit.all()
        for h in range(2):
            bad = hit if h == 1 else np.zeros(n, bool)
            got, gl = o[0, h].cpu().double().numpy(), lse[0, h].cpu().double().numpy()
            assert np.isnan(got[bad]).all() and np.isnan(gl[bad]).all(), (name, h)
            f64 = lambda x: x[0, h].double().numpy()  # noqa: E731
            z, _ = R.scores(f64(base["q"]), f64(base["k"]), p.scale, cap, float(np.float32(slopes[h])), i, i)
            w, wl, tol, lt = R.forward(f64(base["q"]), f64(base["k"]), f64(base["v"]), mask, z)
            assert (np.abs(got - w) <= tol)[~bad].all() and (np.abs(gl - wl) <= lt)[~bad].all(), (name, h)
        dq, dk, dv = backward(t, o, lse)
        assert bool(torch.isnan(dq[0, 1, torch.from_numpy(hit).cuda()]).all())
        seen = mask[hit].any(axis=0)  # keys that such a row attends
        for g in (dk, dv):
            assert bool(torch.isnan(g[0, 1, torch.from_numpy(seen).cuda()]).all())
            assert bool(torch.isfinite(g[0, 0]).all())
        assert bool(torch.isfinite(dq[0, 0]).all())
        if name == "q":
            assert bool(torch.isfinite(dq[0, 1, torch.from_numpy(~hit).cuda()]).all())
        sp.spattn_check(plan)


def test_fp8_codes_of_nan():
    p = _problem(200, head_dim=128)
    plan = sp.Plan.from_problem(p)
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    q8, qd = sp.quantize_fp8(t["q"])
    k8, kd = sp.quantize_fp8(t["k"])
    want, _ = sp.spattn_fwd_fp8(q8, k8, qd, kd, t["v"], plan)
    q8[0, 0, 33, 5] = 0x7F
    o, lse = sp.spattn_fwd_fp8(q8, k8, qd, kd, t["v"], plan)
    assert bool(torch.isnan(o[0, 0, 33]).all()) and bool(torch.isnan(lse[0, 0, 33]))
    o[0, 0, 33] = want[0, 0, 33]
    assert torch.equal(o, want)


@pytest.mark.parametrize("cap", [0.0, 30.0, 90.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n,kv,max_kv", [(1, 777, 777), (1, 9000, 9000), (1, 9000, 1 << 20), (90, 5000, 5000), (5, 40, 40)])
def test_rows_over_a_cache(n, kv, max_kv, bias, cap):
    heads, ps = 4, 32
    gen = torch.Generator().manual_seed(kv)
    pages = -(-kv // ps)
    q = torch.randn((n, heads, 128), generator=gen).bfloat16()
    cache = [torch.randn((pages, ps, 2, 128), generator=gen).bfloat16() for _ in range(2)]
    slopes = [0.01, 0.002, 0.0, 0.1]
    paged = sp.PagedPlan(heads=heads, kv_heads=2, head_dim=128, page_slots=ps, max_seqs=1, max_q=n, max_kv=max_kv,
                         softcap=cap, slopes=torch.tensor(slopes).cuda() if bias else None)
    table = torch.arange(pages, dtype=torch.int32)[None].cuda()
    start, lens = torch.tensor([0, n], dtype=torch.int32).cuda(), torch.tensor([kv], dtype=torch.int32).cuda()

    def run(q, k):
        o, lse = sp.spattn_paged_fwd(q.cuda(), k.cuda(), cache[1].cuda(), table, start, lens, paged)
        sp.spattn_paged_check(paged)
        return o.cpu().double().numpy(), lse.cpu().double().numpy()

    rows = [x.double().numpy().reshape(-1, 2, 128)[:kv] for x in cache]
    w, wl, tol, lt = R.paged(q.double().numpy(), *rows, kv, 128 ** -0.5, cap, [float(np.float32(s)) for s in slopes] if bias else None)

    def check(o, lse, bad):
        assert np.isnan(o[bad]).all() and np.isnan(lse[bad]).all()
        assert (np.abs(o - w) <= tol)[~bad].all() and (np.abs(lse - wl) <= lt)[~bad].all()

    bad = np.zeros((n, heads), bool)
    bad[n // 2, 1] = True
    qn = q.clone()
    qn[n // 2, 1, 7] = NAN
    check(*run(qn, cache[0]), bad)
    # a damaged slot: of the first K/V head, the first position, or the last one, which only the last token attends
    for at in (0, kv - 1):
        kn = cache[0].clone()
        kn[at // ps, at % ps, 0, 99] = NAN
        bad = np.zeros((n, heads), bool)
        bad[kv - n + np.arange(n) >= at, :2] = True
        check(*run(q, kn), bad)
    # every key of a K/V head, in every range of the keys
    kn = cache[0].clone()
    kn[:, :, 1, 0] = NAN
    bad = np.zeros((n, heads), bool)
    bad[:, 2:] = True
    check(*run(q, kn), bad)
