"""Scored attention (cap, bias, document and position masks) against the fp64
oracle, element by element, with the bounds the oracle derives from the
roundings to bf16 (oracle/operators.py)."""

import dataclasses
import os

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
import oracle
from oracle import operators as R
from workloads import configs as W

pytestmark = pytest.mark.gpu


def _score_arrays(p, kind, seed):
    """Per-slot arrays of a masking kind: dict of int32 NumPy arrays."""
    rng = np.random.default_rng(seed)
    nq, nk = p.q_slots, p.kv_slots
    qp, kp = np.arange(nq), np.arange(nk)
    if kind == "none":
        return {}
    if kind == "bias":
        return dict(q_pos=qp - 40, k_pos=kp - 60)
    if kind == "causal":
        return dict(q_pos=qp, k_pos=kp, q_last=qp)
    if kind == "prefix":
        return dict(q_pos=qp, k_pos=kp, q_last=np.maximum(qp, 90))
    if kind == "frames":  # few distinct positions, in an order unlike the slots'
        qp, kp = rng.integers(0, 5, nq), rng.integers(0, 5, nk)
        return dict(q_pos=qp, k_pos=kp, q_last=qp)
    if kind == "docs":  # runs of 1 .. 60 slots, some slots without a document
        def runs(n):
            d = np.repeat(np.arange(n), rng.integers(1, 61, n))[:n]
            d[rng.random(n) < 0.05] = -1
            return d
        return dict(q_doc=runs(nq), k_doc=runs(nk))
    if kind == "mixed":  # documents in no order, causal inside, positions far out, rows that attend nothing
        qp, kp = rng.integers(-2 ** 24, 2 ** 24, nq), rng.integers(-2 ** 24, 2 ** 24, nk)
        last = np.where(rng.random(nq) < 0.1, -2 ** 31, np.where(rng.random(nq) < 0.2, 2 ** 31 - 1, qp))
        return dict(q_pos=qp, k_pos=kp, q_last=last, q_doc=rng.integers(-1, 3, nq), k_doc=rng.integers(-1, 3, nk))
    raise KeyError(kind)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int64).astype(np.int32))).cuda()


def _score(arrays, cap, slopes):
    return sp.Score(softcap=cap, slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda(),
                    **{n: _i32(a) for n, a in arrays.items()})


def _run(p, t, plan, sc):
    dev = {k: v.cuda() for k, v in t.items()}
    o, lse = sp.spattn_fwd_scored(dev["q"], dev["k"], dev["v"], plan, sc)
    dq, dk, dv = sp.spattn_bwd_scored(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], plan, sc)
    sp.spattn_check(plan)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _close(got, want, tol, what):
    assert np.isfinite(got).all(), what
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) / np.maximum(tol, 1e-30)).max()))


def _check(p, t, out, arrays, cap, slopes):
    f64 = lambda x: x.cpu().double().numpy()  # noqa: E731
    group = p.heads // p.n_kv_heads
    for b in range(p.batch):
        pick = lambda n: None if n not in arrays else (arrays[n][b] if np.ndim(arrays[n]) == 2 else arrays[n])  # noqa: E731
        acc = {}
        for h in range(p.heads):
            hk = h // group
            A = oracle.allowed_groups(p.row_ptr, p.kv_groups, p.n_q_groups, p.n_kv_groups, p.graph_head(b, h))
            M = R.score_mask(oracle.token_mask(p.q_group, p.kv_group, A), pick("k_pos"), pick("q_last"), pick("q_doc"),
                             pick("k_doc"))
            q, do = f64(t["q"][b, h]), f64(t["do"][b, h])
            k, v = f64(t["k"][b, hk]), f64(t["v"][b, hk])
            # padded rows hold a sentinel that no result may see; keep it out of the bounds too
            q, do = (np.where((p.q_group >= 0)[:, None], x, 0.0) for x in (q, do))
            k, v = (np.where((p.kv_group >= 0)[:, None], x, 0.0) for x in (k, v))
            z, f = R.scores(q, k, p.scale, cap, 0.0 if slopes is None else float(np.float32(slopes[h])), pick("q_pos"),
                            pick("k_pos"))
            o, lse, o_tol, lse_tol = R.forward(q, k, v, M, z)
            some = M.any(axis=1)
            go, gl = f64(out["o"][b, h]), f64(out["lse"][b, h])
            _close(go, o, o_tol, ("o", b, h))
            assert (gl[~some] == -np.inf).all() and (go[~some] == 0).all()
            _close(gl[some], lse[some], lse_tol[some], ("lse", b, h))
            g = R.backward(q, k, v, do, M, z, f, p.scale)
            _close(f64(out["dq"][b, h]), *g["dq"], ("dq", b, h))
            assert (f64(out["dq"][b, h])[~some] == 0).all()
            for n in ("dk", "dv"):
                val, tol = acc.setdefault((n, hk), [0.0, 0.0])
                acc[(n, hk)] = [val + g[n][0], tol + g[n][1]]
        for (n, hk), (val, tol) in acc.items():
            got = f64(out[n][b, hk])
            _close(got, val, tol, (n, b, hk))
            assert (got[p.kv_group < 0] == 0).all()


# small caps take the tanh itself (scores beyond half the cap), larger ones its
# polynomial, 60 is above the fixed-reference limit, 1e6 is a cap that does nothing
CASES = [
    ("tiny", "causal", 2.0, None), ("tiny", "bias", 0.0, 0.3), ("tiny_vsa", "docs", 30.0, None),
    ("tiny_svg2", "mixed", 0.0, None), ("tiny_svg2", "mixed", 5.0, None), ("tiny_svg2", "prefix", 60.0, 0.05),
    ("tiny_d128", "causal", 30.0, -0.02), ("tiny_d128", "docs", 0.0, 0.1), ("tiny_hedge", "frames", 20.0, 0.5),
    ("tiny_empty", "frames", 0.0, None), ("tiny_onekey", "causal", 1.0, 0.01), ("tiny_nokeys", "docs", 50.0, None),
    ("tiny_gqa", "prefix", 15.0, 0.2), ("tiny_mqa", "docs", 0.0, 0.7), ("tiny_bgraph", "frames", 30.0, 0.1),
    ("tiny_svg2", "none", 1e6, None), ("tiny_d128", "none", 60.0, None), ("tiny_gqa", "mixed", 3.0, 1e-6),
]


@pytest.mark.parametrize("name,kind,cap,slope", CASES)
def test_scored_parity(name, kind, cap, slope):
    p = W.make_problem(name)
    t = W.make_tensors(p)
    arrays = _score_arrays(p, kind, len(name) + int(cap))
    if slope is not None and "q_pos" not in arrays:
        arrays.update(q_pos=np.arange(p.q_slots), k_pos=np.arange(p.kv_slots))
    slopes = None if slope is None else slope * 2.0 ** -np.arange(p.heads)
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, cap, slopes))
    _check(p, t, out, arrays, cap, slopes)


@pytest.mark.parametrize("pack", ["route64", "split", "slot"])
@pytest.mark.parametrize("kind,cap", [("mixed", 0.0), ("docs", 30.0), ("causal", 70.0)])
def test_scored_parity_of_forced_packings(pack, kind, cap, monkeypatch):
    monkeypatch.setenv("SPATTN_PLAN_PACK", pack)
    p = W.make_problem("tiny_svg2")
    t = W.make_tensors(p)
    arrays = _score_arrays(p, kind, 5)
    slopes = [0.03, 0.5] if kind != "docs" else None
    if kind == "mixed":
        slopes = None  # its positions are far apart: every weight but one would vanish
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, cap, slopes))
    _check(p, t, out, arrays, cap, slopes)


def _token_problem(n, heads=1, head_dim=64, batch=1, kv_heads=0):
    """n tokens in 64-slot blocks, every block pair listed."""
    nb = -(-n // 64)
    group = (np.arange(n) // 64).astype(np.int32)
    rows = np.arange(0, heads * nb * nb + 1, nb, dtype=np.int64)
    return W.Problem(f"tokens{n}", batch, heads, head_dim, group, group.copy(), nb, nb, rows,
                     np.tile(np.arange(nb, dtype=np.int32), heads * nb), 21000 + n, kv_heads=kv_heads)


@pytest.mark.parametrize("n", [1, 2, 15, 17, 63, 65, 129, 200])
@pytest.mark.parametrize("cap", [0.0, 25.0])
def test_lengths(n, cap):
    p = _token_problem(n, heads=2, head_dim=128, kv_heads=1)
    t = W.make_tensors(p)
    arrays = _score_arrays(p, "causal", 0)
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, cap, None))
    _check(p, t, out, arrays, cap, None)


@pytest.mark.parametrize("cap", [0.0, 20.0, 80.0])
def test_single_key_rows_are_exact(cap):
    """Documents of one token: O = v, and dQ = dK = 0 exactly."""
    p = _token_problem(150)
    t = W.make_tensors(p)
    arrays = dict(q_doc=np.arange(150), k_doc=np.arange(150))
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, cap, None))
    assert torch.equal(out["o"].cpu(), t["v"])
    assert int(out["dq"].count_nonzero()) == 0 and int(out["dk"].count_nonzero()) == 0
    _check(p, t, out, arrays, cap, None)


def test_batched_arrays():
    p = dataclasses.replace(W.make_problem("tiny_bgraph"))
    t = W.make_tensors(p)
    one = [_score_arrays(p, "docs", s) for s in (1, 2)]
    arrays = {n: np.stack([o[n] for o in one]) for n in one[0]}
    rng = np.random.default_rng(0)
    arrays.update(q_pos=rng.integers(0, 99, (2, p.q_slots)), k_pos=rng.integers(0, 99, (2, p.kv_slots)))
    arrays["q_last"] = arrays["q_pos"]
    slopes = [0.01, 0.2]
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, 12.0, slopes))
    _check(p, t, out, arrays, 12.0, slopes)


def test_neutral_score_is_the_plain_call():
    p = W.make_problem("tiny_svg2")
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    plan = sp.Plan.from_problem(p)
    o, lse = sp.spattn_fwd(t["q"], t["k"], t["v"], plan)
    a = sp.spattn_bwd(t["q"], t["k"], t["v"], o, lse, t["do"], plan)
    sc = sp.Score()
    o2, lse2 = sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc)
    b = sp.spattn_bwd_scored(t["q"], t["k"], t["v"], o, lse, t["do"], plan, sc)
    for x, y in zip((o, lse) + a, (o2, lse2) + b):
        assert torch.equal(x, y)


def test_large_scores_and_values():
    """Scores far beyond the cap (tanh saturates: every gradient of Q and K vanishes) and large values."""
    p = _token_problem(130, head_dim=64)
    t = W.make_tensors(p)
    t["q"], t["v"] = t["q"] * 300, t["v"] * 1e4
    arrays = _score_arrays(p, "causal", 0)
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, 4.0, None))
    _check(p, t, out, arrays, 4.0, None)


def _lift(t):
    """Adds +-96 * 8 * scale (+-96 for head_dim 64, +-68 for 128, exact in fp32) to every score of two
    thirds of the rows: their LSE leaves +-55, the others' stays.  All scores stay below 2^7, for which the
    oracle's fp32 share (2^-24 * 2^7 * 8 = 2^-14 of a weight) is what it allows."""
    t["k"][..., 0] = 8.0
    rows = torch.arange(t["q"].shape[2]) % 3
    t["q"][..., 0] = torch.where(rows == 0, 96.0, torch.where(rows == 1, -96.0, 0.0)).to(t["q"].dtype)


@pytest.mark.parametrize("n,head_dim", [(1, 64), (40, 64), (65, 128), (130, 64), (200, 128)])
@pytest.mark.parametrize("cap", [0.0, 250.0])
@pytest.mark.parametrize("kind", ["causal", "docs"])
def test_rows_of_extreme_scores(n, head_dim, cap, kind):
    p = _token_problem(n, heads=2, head_dim=head_dim)
    t = W.make_tensors(p)
    _lift(t)
    arrays = _score_arrays(p, kind, n)
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, cap, None))
    _check(p, t, out, arrays, cap, None)


@pytest.mark.parametrize("pack", ["route64", "split", "slot"])
def test_rows_of_extreme_scores_in_forced_packings(pack, monkeypatch):
    monkeypatch.setenv("SPATTN_PLAN_PACK", pack)
    p = W.make_problem("tiny_svg2")
    t = W.make_tensors(p)
    kept = {n: t[n].clone() for n in ("q", "k")}
    _lift(t)
    for n, group in (("q", p.q_group), ("k", p.kv_group)):  # the padded rows keep their sentinel
        pad = torch.from_numpy(group < 0)
        t[n][:, :, pad] = kept[n][:, :, pad]
    arrays = _score_arrays(p, "prefix", 2)
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, 0.0, None))
    _check(p, t, out, arrays, 0.0, None)


@pytest.mark.parametrize("n", [5, 70, 150])
def test_keys_all_far_away(n):
    """A bias of 100 and more on every key of every row (one head) leaves weights, O and gradients whole."""
    p = _token_problem(n, heads=2)
    t = W.make_tensors(p)
    arrays = dict(q_pos=np.arange(n) % 32 + 400, k_pos=np.arange(n) % 32, q_last=np.arange(n))
    slopes = [0.25, 0.001]
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, 0.0, slopes))
    _check(p, t, out, arrays, 0.0, slopes)


@pytest.mark.parametrize("cap", [1e-40, 1e-20, 1e-6, 1e30])
def test_extreme_caps(cap):
    """Caps whose scaled coefficients leave fp32; queries of zeros (scores of exactly 0) among the rows."""
    p = _token_problem(90, head_dim=64)
    t = W.make_tensors(p)
    t["q"][:, :, 20:30] = 0
    arrays = _score_arrays(p, "causal", 0)
    dev = {k: v.cuda() for k, v in t.items()}
    plan, sc = sp.Plan.from_problem(p), _score(arrays, cap, None)
    o, lse = sp.spattn_fwd_scored(dev["q"], dev["k"], dev["v"], plan, sc)
    grads = sp.spattn_bwd_scored(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], plan, sc)
    assert all(bool(torch.isfinite(x).all()) for x in (o, lse) + tuple(grads))
    f64 = lambda x: x[0, 0].cpu().double().numpy()  # noqa: E731
    mask = R.score_mask(np.ones((90, 90), bool), arrays["k_pos"], arrays["q_last"])
    z, _ = R.scores(f64(t["q"]), f64(t["k"]), p.scale, float(np.float32(cap)) or cap)
    want, wl, tol, lt = R.forward(f64(t["q"]), f64(t["k"]), f64(t["v"]), mask, z)
    _close(f64(o), want, tol, "o")
    _close(f64(lse), wl, lt, "lse")


def test_device_replan_keeps_the_score():
    p = W.make_problem("tiny_vsa")
    t = W.make_tensors(p)
    plan = sp.Plan.from_problem(p)
    rng = np.random.default_rng(9)
    row_ptr, cols = W.vsa_graph(12, 2, 6, rng)
    plan.set_graph_device(torch.from_numpy(row_ptr).cuda(), torch.from_numpy(cols).cuda())
    p2 = dataclasses.replace(p, row_ptr=row_ptr, kv_groups=cols)
    arrays = _score_arrays(p, "prefix", 0)
    out = _run(p2, t, plan, _score(arrays, 10.0, [0.1, 0.0]))
    _check(p2, t, out, arrays, 10.0, [0.1, 0.0])


@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_capture_replay_streams_and_repeats(cap):
    """A captured step replayed with new inputs equals an eager one on another stream, bit for bit."""
    p = W.make_problem("tiny_gqa")
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    arrays = _score_arrays(p, "prefix", 3)
    sc = _score(arrays, cap, [0.1, 0.2, 0.0, 0.4])
    plan = sp.Plan.from_problem(p)

    def step():
        o, lse = sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc)
        return (o, lse) + tuple(sp.spattn_bwd_scored(t["q"], t["k"], t["v"], o, lse, t["do"], plan, sc))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    t["q"].copy_(t["q"].flip(2))
    t["do"].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in captured]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    side.synchronize()
    for x, y in zip(got, eager):
        assert torch.equal(x, y)
    for _ in range(5):
        for x, y in zip(eager, step()):
            assert torch.equal(x, y)
    sp.spattn_check(plan)


def test_two_plans_on_two_streams():
    p = W.make_problem("tiny_svg2")
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    sc = [_score(_score_arrays(p, k, 1), c, None) for k, c in (("prefix", 0.0), ("docs", 30.0))]
    plans = [sp.Plan.from_problem(p) for _ in sc]
    want = [sp.spattn_fwd_scored(t["q"], t["k"], t["v"], pl, s) for pl, s in zip(plans, sc)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sc]
    got = []
    for _ in range(10):
        got.append([sp.spattn_fwd_scored(t["q"], t["k"], t["v"], pl, s, stream=st)
                    for pl, s, st in zip(plans, sc, streams)])
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_against_differences():
    """The library's dQ, dK, dV along random directions against central differences of its own forward's
    loss in fp64 (the oracle's loss at the bf16 inputs)."""
    p = _token_problem(70)
    t = W.make_tensors(p)
    arrays, cap, slopes = _score_arrays(p, "causal", 0), 3.0, [0.05]
    out = _run(p, t, sp.Plan.from_problem(p), _score(arrays, cap, slopes))
    x = {n: t[n][0, 0].double().numpy() for n in ("q", "k", "v", "do")}
    mask = R.score_mask(np.ones((70, 70), bool), arrays["k_pos"], arrays["q_last"])
    rng = np.random.default_rng(4)

    def loss(a):
        z, _ = R.scores(a["q"], a["k"], p.scale, cap, float(np.float32(0.05)), arrays["q_pos"], arrays["k_pos"])
        return float((R.forward(a["q"], a["k"], a["v"], mask, z)[0] * x["do"]).sum())

    for n in ("q", "k", "v"):
        d = rng.standard_normal(x[n].shape)
        h = 1e-5
        num = (loss({**x, n: x[n] + h * d}) - loss({**x, n: x[n] - h * d})) / (2 * h)
        z, f = R.scores(x["q"], x["k"], p.scale, cap, float(np.float32(0.05)), arrays["q_pos"], arrays["k_pos"])
        tol = R.backward(x["q"], x["k"], x["v"], x["do"], mask, z, f, p.scale)["d" + n][1]
        got = float((out["d" + n][0, 0].cpu().double().numpy() * d).sum())
        assert abs(got - num) <= float((tol * np.abs(d)).sum()) + 1e-6 * abs(num), n


def test_another_current_device_is_refused(monkeypatch):
    p = W.make_problem("tiny")
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    plan = sp.Plan.from_problem(p)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sp.Score(softcap=1.0))


def test_wrong_devices_and_shapes_are_refused():
    p = W.make_problem("tiny")
    t = {k: v.cuda() for k, v in W.make_tensors(p).items()}
    plan = sp.Plan.from_problem(p)
    pos = torch.arange(768, dtype=torch.int32).cuda()

    def call(sc, **over):
        a = {**t, **over}
        return sp.spattn_fwd_scored(a["q"], a["k"], a["v"], plan, sc)

    for sc in (sp.Score(slopes=torch.ones(3).cuda(), q_pos=pos, k_pos=pos), sp.Score(q_last=pos[:-1], k_pos=pos),
               sp.Score(q_last=pos.long(), k_pos=pos), sp.Score(q_last=pos.cpu(), k_pos=pos),
               sp.Score(q_last=pos, k_pos=pos[None]), sp.Score(q_doc=torch.stack([pos, pos], 1)[:, 0], k_doc=pos)):
        with pytest.raises(ValueError):
            call(sc)
    with pytest.raises(ValueError):
        call(sp.Score(softcap=1.0), q=t["q"].float())
    with pytest.raises(ValueError):
        call(sp.Score(softcap=1.0), k=t["k"].transpose(2, 3).contiguous().transpose(2, 3))
    for sc in (sp.Score(softcap=-1.0), sp.Score(softcap=float("nan")), sp.Score(softcap=float("inf")),
               sp.Score(slopes=torch.ones(2).cuda()), sp.Score(q_last=pos), sp.Score(q_doc=pos),
               sp.Score(slopes=torch.ones(2).cuda(), q_pos=pos)):
        with pytest.raises(sp.SpattnError) as e:
            call(sc)
        assert e.value.status == sp.SPATTN_ERR_INVALID_ARG
    torch.cuda.synchronize()
    sp.spattn_check(plan)
