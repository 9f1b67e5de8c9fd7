"""Scored attention with more work items than the GPU runs at once: persistent CTAs that take
several items (column lines, barriers and the item queue carried over), more items than
are ordered by length, and lists of many steps. A few (batch entry, K/V head)s of each
problem are checked against the fp64 oracle (oracle/operators.py), the rest by running the
call again on those alone."""

import dataclasses

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
from oracle import operators as R
from workloads import configs as W

pytestmark = pytest.mark.gpu

SMS, ORDERED = 148, 32 * 148  # SMs, and items up to which lists are ordered by length


def _problem(n, batch, heads, kv_heads, head_dim, lists):
    """n tokens in 64-slot blocks; ``lists``: every block, or those up to the own one."""
    nb = -(-n // 64)
    group = (np.arange(n) // 64).astype(np.int32)
    rows = [list(range(nb if lists == "all" else a + 1)) for a in range(nb)] * heads
    return W.Problem(f"large{n}", batch, heads, head_dim, group, group.copy(), nb, nb,
                     np.cumsum([0] + [len(r) for r in rows]).astype(np.int64), np.concatenate(rows).astype(np.int32), 31,
                     kv_heads=kv_heads)


def _arrays(n, kind, batch, rng):
    i = np.arange(n)
    if kind == "causal":
        return dict(q_pos=i, k_pos=i, q_last=i)
    if kind == "prefix":
        return dict(q_pos=i, k_pos=i, q_last=np.maximum(i, n // 3))
    if kind == "docs":  # other documents in every batch entry
        d = np.stack([np.repeat(np.arange(n), rng.integers(1, 90, n))[:n] for _ in range(batch)])
        return dict(q_doc=d, k_doc=d)
    return dict(q_pos=i, k_pos=i)


def _score(arrays, cap, slopes):
    gpu = {k: torch.from_numpy(np.ascontiguousarray(v).astype(np.int32)).cuda() for k, v in arrays.items()}
    return sp.Score(softcap=cap, slopes=None if slopes is None else torch.from_numpy(slopes).cuda(), **gpu)


def _run(t, plan, sc):
    o, lse = sp.spattn_fwd_scored(t["q"], t["k"], t["v"], plan, sc)
    out = dict(zip(("dq", "dk", "dv"), sp.spattn_bwd_scored(t["q"], t["k"], t["v"], o, lse, t["do"], plan, sc)))
    sp.spattn_check(plan)
    return dict(out, o=o, lse=lse)


CASES = [
    # tokens, batch, heads, kv heads, head dim, lists, masks, cap, slope
    (130, 10, 40, 40, 64, "all", "causal", 20.0, None),
    (130, 40, 40, 8, 128, "all", "docs", 0.0, None),
    (300, 15, 48, 16, 64, "causal", "causal", 0.0, 0.05),
    (300, 7, 32, 32, 128, "all", "prefix", 8.0, 0.02),
    (64, 120, 40, 40, 64, "all", "causal", 0.0, None),  # 4800 items a pass: more than are ordered
    (60, 240, 40, 20, 64, "all", "docs", 30.0, None),
    (1500, 4, 28, 4, 64, "causal", "prefix", 0.0, None),  # lists of up to 24 steps
    (1100, 3, 24, 24, 128, "all", "docs", 15.0, None),
    (1300, 2, 32, 8, 128, "all", "none", 25.0, 0.01),
]


@pytest.mark.parametrize("n,batch,heads,kv,d,lists,kind,cap,slope", CASES)
def test_parity(n, batch, heads, kv, d, lists, kind, cap, slope):
    p = _problem(n, batch, heads, kv, d, lists)
    rng = np.random.default_rng(n + heads)
    arrays = _arrays(n, kind, batch, rng)
    slopes = None if slope is None else (slope * 2.0 ** -(np.arange(heads) % 7)).astype(np.float32)
    gen = torch.Generator(device="cuda").manual_seed(n)
    rand = lambda h: torch.randn((batch, h, n, d), generator=gen, device="cuda").bfloat16()  # noqa: E731
    t = {"q": rand(heads), "k": rand(kv), "v": rand(kv), "do": rand(heads)}
    plan = sp.Plan.from_problem(p)
    items = plan.stats()["n_work_dkdv"], plan.stats()["n_work_fwd"]
    assert min(items) > (ORDERED if n < 128 else 4 * SMS if n < 1000 else SMS)
    sc = _score(arrays, cap, slopes)
    out = _run(t, plan, sc)
    again = _run(t, plan, sc)
    for name in out:
        assert torch.equal(out[name], again[name]), name
        assert not bool(torch.isnan(out[name]).any())
    group = heads // kv
    block = np.arange(n) // 64
    graph = np.ones((n, n), bool) if lists == "all" else block[None, :] <= block[:, None]
    pick = [(int(b), int(h)) for b, h in zip(rng.integers(0, batch, 3), rng.integers(0, kv, 3))] + [(batch - 1, kv - 1)]
    for b, hk in pick:
        row = lambda k: None if k not in arrays else arrays[k][b] if arrays[k].ndim == 2 else arrays[k]  # noqa: E731
        M = R.score_mask(graph, row("k_pos"), row("q_last"), row("q_doc"), row("k_doc"))
        f64 = lambda x, h: x[b, h].cpu().double().numpy()  # noqa: E731
        acc = {"dk": [0.0, 0.0], "dv": [0.0, 0.0]}
        for h in range(hk * group, (hk + 1) * group):
            q, k, v, do = f64(t["q"], h), f64(t["k"], hk), f64(t["v"], hk), f64(t["do"], h)
            z, f = R.scores(q, k, d ** -0.5, cap, 0.0 if slopes is None else float(slopes[h]), row("q_pos"), row("k_pos"))
            o, lse, o_tol, lse_tol = R.forward(q, k, v, M, z)
            assert (np.abs(f64(out["o"], h) - o) <= o_tol).all(), (b, h)
            assert (np.abs(f64(out["lse"], h) - lse) <= lse_tol).all(), (b, h)
            g = R.backward(q, k, v, do, M, z, f, d ** -0.5, M.sum(axis=1) <= 16)
            assert (np.abs(f64(out["dq"], h) - g["dq"][0]) <= g["dq"][1]).all(), (b, h)
            for name in acc:
                acc[name] = [acc[name][0] + g[name][0], acc[name][1] + g[name][1]]
        for name, (val, tol) in acc.items():
            assert (np.abs(f64(out[name], hk) - val) <= tol).all(), (name, b, hk)
    # the other heads: the same bits from a call over one batch entry
    one = dataclasses.replace(p, batch=1)
    plan1 = sp.Plan.from_problem(one)
    for b in {0, batch // 2, pick[0][0]}:
        s1 = _score({k: v[b] if v.ndim == 2 else v for k, v in arrays.items()}, cap, slopes)
        alone = _run({k: v[b:b + 1].contiguous() for k, v in t.items()}, plan1, s1)
        for name in out:
            assert torch.equal(out[name][b:b + 1], alone[name]), (name, b)
