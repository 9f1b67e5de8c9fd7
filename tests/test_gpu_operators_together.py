"""The operators as a model runs them: rotary positions, scored attention and
its gradients back to the projection; and decoding from a paged cache that
gives what the full forward gives."""

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
from oracle import operators as R

pytestmark = pytest.mark.gpu

B, H, HK, D, N, CAP, PREFIX = 1, 4, 2, 64, 150, 20.0, 30


def _setup():
    gen = torch.Generator().manual_seed(11)
    qkv = torch.randn((B, N, H + 2 * HK, D), generator=gen).bfloat16().cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    freqs, mscale = sp.rope_freqs(D // 2, scaling="yarn", factor=4.0, original_slots=64)
    nb = -(-N // 64)
    group = (np.arange(N) // 64).astype(np.int32)
    plan = sp.Plan(group, group, nb, nb, np.arange(0, H * nb * nb + 1, nb), np.tile(np.arange(nb), H * nb), batch=B,
                   heads=H, kv_heads=HK, head_dim=D)
    slopes = torch.tensor([0.2, 0.1, 0.05, 0.0]).cuda()
    return qkv, pos, freqs, mscale, plan, slopes


def test_training_step_through_all_of_them():
    qkv, pos, freqs, mscale, plan, slopes = _setup()
    sc = sp.Score(softcap=CAP, slopes=slopes, q_pos=pos, k_pos=pos, q_last=torch.clamp(pos, min=PREFIX - 1))
    q0, k0 = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + HK].transpose(1, 2)
    v = qkv[:, :, H + HK:].transpose(1, 2).contiguous()
    q, k = sp.rope(q0, k0, pos, freqs, mscale=mscale)
    o, lse = sp.spattn_fwd_scored(q, k, v, plan, sc)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(12)).bfloat16().cuda()
    dq, dk, dv = sp.spattn_bwd_scored(q, k, v, o, lse, do, plan, sc)
    dqkv = torch.zeros_like(qkv)
    sp.rope_bwd(dq, dk, pos, freqs, mscale=mscale, dq=dqkv[:, :, :H].transpose(1, 2),
                dk=dqkv[:, :, H:H + HK].transpose(1, 2))
    dqkv[:, :, H + HK:] = dv.transpose(1, 2)
    sp.spattn_check(plan)
    # the whole step in fp64 by autograd, from the same bf16 projection
    x = qkv.cpu().double().requires_grad_()
    ang = pos.cpu().double()[:, None] * freqs.cpu()

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        c, s = mscale * torch.cos(ang), mscale * torch.sin(ang)
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    qq, kk = turn(x[:, :, :H].transpose(1, 2)), turn(x[:, :, H:H + HK].transpose(1, 2))
    vv = x[:, :, H + HK:].transpose(1, 2)
    kk, vv = kk.repeat_interleave(H // HK, 1), vv.repeat_interleave(H // HK, 1)
    i = torch.arange(N)
    z = CAP * torch.tanh(qq @ kk.mT / D ** 0.5 / CAP) - slopes.cpu().double()[:, None, None] * (i[:, None] - i).abs()
    z = z.masked_fill(i > torch.clamp(i, min=PREFIX - 1)[:, None], -1e30)
    out = torch.softmax(z, -1) @ vv
    (out * do.cpu().double()).sum().backward()
    # roundings on the way of each value, of 2^-8 at most and independent: Q and K, the
    # weights or dS, O in Delta, dQ, and the result: five of them in the 2-norm
    tol = 5 ** 0.5 * 2.0 ** -8
    rel = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    assert rel(o, out.detach()) <= tol
    for name, part in (("q", slice(0, H)), ("k", slice(H, H + HK)), ("v", slice(H + HK, None))):
        assert rel(dqkv[:, :, part], x.grad[:, :, part]) <= tol, name


@pytest.mark.parametrize("chunks", [[150], [100, 1, 1, 48], [1] * 6])
def test_serving_from_a_cache_matches_the_full_forward(chunks):
    """Prefill and decode over a paged cache, token rows written after their rotation, against the scored
    forward over the whole causal sequence on the same rotated Q, K, V."""
    qkv, pos, freqs, mscale, plan, slopes = _setup()
    n = sum(chunks)
    sc = sp.Score(softcap=CAP, slopes=slopes, q_pos=pos, k_pos=pos, q_last=pos)
    q, k = sp.rope(qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + HK].transpose(1, 2), pos, freqs, mscale=mscale)
    v = qkv[:, :, H + HK:].transpose(1, 2).contiguous()
    full, full_lse = sp.spattn_fwd_scored(q, k, v, plan, sc)
    ps = 16
    pages = -(-n // ps)
    table = torch.randperm(pages + 2, generator=torch.Generator().manual_seed(1))[:pages].int().cuda()[None]
    kc, vc = (torch.full((pages + 2, ps, HK, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    paged = sp.PagedPlan(heads=H, kv_heads=HK, head_dim=D, page_slots=ps, max_seqs=1, max_q=max(chunks), max_kv=n,
                         softcap=CAP, slopes=slopes)
    at = 0
    for c in chunks:
        rows = slice(at, at + c)
        part = qkv[:, rows]
        qs, ks = sp.rope(part[:, :, :H].transpose(1, 2), part[:, :, H:H + HK].transpose(1, 2), pos[rows].contiguous(),
                         freqs, mscale=mscale)
        assert torch.equal(ks, k[:, :, rows])
        i = torch.arange(at, at + c).cuda()
        where = (table[0].long()[i // ps], i % ps)
        kc[where], vc[where] = ks[0].transpose(0, 1), part[0, :, H + HK:]
        o, lse = sp.spattn_paged_fwd(qs[0].transpose(0, 1), kc, vc, table,
                                     torch.tensor([0, c], dtype=torch.int32).cuda(),
                                     torch.tensor([at + c], dtype=torch.int32).cuda(), paged)
        sp.spattn_paged_check(paged)
        want = full[0, :, rows].transpose(0, 1).double()
        # both round weights and results: each within 2^-8 (sum P |v| + |O|) of the exact value, |v| <= 5
        assert float((o.double() - want).abs().max()) <= 2 * 2.0 ** -8 * 2 * float(v.abs().max())
        assert float((o.double() - want).norm() / want.norm()) <= 2 * 2.0 ** -8
        assert float((lse - full_lse[0, :, rows].T).abs().max()) <= 2 * (2.0 ** -15 + 2.0 ** -20 * 20)
        at += c


@pytest.mark.parametrize("n", [9, 70, 150])
def test_results_do_not_depend_on_what_ran_before(n):
    """Tiles with rows and columns that nothing fills (tensor memory then holds what an earlier kernel left
    there) give the same bits after kernels that left zeros and after kernels that left large scores."""
    gen = torch.Generator().manual_seed(n)

    def problem(tokens, heads):
        nb = -(-tokens // 64)
        group = (np.arange(tokens) // 64).astype(np.int32)
        plan = sp.Plan(group, group, nb, nb, np.arange(0, heads * nb * nb + 1, nb), np.tile(np.arange(nb), heads * nb),
                       batch=1, heads=heads, head_dim=64)
        t = [torch.randn((1, heads, tokens, 64), generator=gen).bfloat16().cuda() for _ in range(4)]
        return plan, t

    def scored(plan, q, k, v, do):
        sc = sp.Score(softcap=20.0)
        o, lse = sp.spattn_fwd_scored(q, k, v, plan, sc)
        return (o, lse) + tuple(sp.spattn_bwd_scored(q, k, v, o, lse, do, plan, sc))

    def paged(cap, tokens, cached, heads, q, kv):
        p = sp.PagedPlan(heads=heads, kv_heads=1, head_dim=64, page_slots=16, max_seqs=1, max_q=tokens, max_kv=cached,
                         softcap=cap)
        pages = -(-cached // 16)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        return sp.spattn_paged_fwd(q, kv[:pages], kv[:pages], i32([list(range(pages))]), i32([0, tokens]), i32([cached]), p)

    plan, x = problem(n, 2)
    wide, y = problem(1024, 40)
    kv = torch.randn((128, 16, 1, 64), generator=gen).bfloat16().cuda()
    one = torch.randn((1, 5, 64), generator=gen).bfloat16().cuda()
    many = torch.randn((32, 128, 64), generator=gen).bfloat16().cuda()
    got = []
    for size in (0.0, 1000.0):
        for f in (lambda: scored(plan, *x), lambda: paged(20.0, 1, n, 5, one, kv), lambda: paged(70.0, 1, n, 5, one, kv)):
            scored(wide, y[0] * size, *y[1:])
            paged(20.0, 32, 2048, 128, many * size, kv)
            got.append(f())
    for a, b in zip(got[:3], got[3:]):
        for u, w in zip(a, b):
            assert torch.equal(u, w)
