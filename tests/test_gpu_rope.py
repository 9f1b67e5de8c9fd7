"""Rotary positions against the fp64 oracle, element by element.

Bound of one element: its rounding to the output type (eps / 2 of it) plus
fp32's part, 8 roundings of 2^-24 on the pair's magnitude (the reduced angle,
sine, cosine, scaling, two products, their sum) with the angle's counted 2 pi times."""

import numpy as np
import pytest
import torch

import block_sparse_attention_bwd_b200 as sp
from oracle import operators as R

pytestmark = pytest.mark.gpu


def _check(got, x, y, rot, interleaved, mscale):
    got, eps = got.cpu().double().numpy(), torch.finfo(got.dtype).eps
    i = np.arange(rot // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    mass = np.zeros_like(y)
    mass[..., lo] = mass[..., hi] = abs(mscale) * (np.abs(x[..., lo]) + np.abs(x[..., hi]))
    tiny = float(torch.finfo(torch.float16).tiny) * eps if eps > 1e-4 else 0.0  # fp16 outputs below its normals
    tol = eps / 2 * np.abs(y) * (1 + eps) + 14 * 2.0 ** -24 * mass + tiny
    assert (got[..., rot:] == x[..., rot:]).all()
    bad = np.abs(got - y) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - y).max()))


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


CASES = [  # B, H, Hk, S, D, rot, interleaved, sections, dtype, mscale, pos rows per batch entry
    (1, 2, 1, 1, 128, 128, False, [64], torch.bfloat16, 1.0, False),
    (2, 4, 2, 33, 128, 128, True, [22, 21, 21], torch.bfloat16, 1.0, False),
    (1, 3, 3, 257, 64, 32, False, [10, 6], torch.float16, 1.2, False),
    (3, 1, 1, 19, 96, 64, True, [32], torch.float32, 0.7, True),
    (1, 5, 1, 40, 80, 74, False, [37], torch.bfloat16, 1.0, False),
    (1, 5, 5, 40, 80, 74, True, [30, 7], torch.float16, 1.0, False),
    (2, 2, 2, 7, 7, 6, True, [3], torch.float32, 1.0, True),
    (1, 2, 2, 9, 13, 10, False, [0, 5, 0], torch.bfloat16, 1.0, False),
    (1, 1, 1, 5, 256, 256, False, [128], torch.float32, 1.0, False),
    (1, 2, 1, 6, 64, 0, False, [0], torch.bfloat16, 1.0, False),
    (1, 1, 1, 3, 1024, 1022, True, [511], torch.float16, 1.0, False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_parity(case, inverse):
    B, H, Hk, S, D, rot, inter, sec, dt, ms, per_batch = case
    q, k = _rand((B, H, S, D), dt, 1), _rand((B, Hk, S, D), dt, 2)
    rng = np.random.default_rng(3)
    pos = rng.integers(-2 ** 31, 2 ** 31, (B, len(sec), S)) if per_batch else rng.integers(-50, 10 ** 5, (len(sec), S))
    freqs = np.concatenate([100.0 ** (-np.arange(n) / max(n, 1)) for n in sec]) if rot else np.zeros(0)
    f = sp.rope_bwd if inverse else sp.rope
    yq, yk = f(q, k, torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(freqs).cuda(), rot_dim=rot,
               interleaved=inter, sections=sec, mscale=ms)
    assert yq.is_contiguous() and yk.is_contiguous() and yq.dtype == dt
    for x, y in ((q, yq), (k, yk)):
        x = x.cpu().double().numpy()
        for b in range(B):
            _check(y[b], x[b], R.rope(x[b], pos[b] if per_batch else pos, freqs, sec, rot, inter, ms, inverse), rot, inter, ms)


def _call_args(S=20, pairs=32):
    return torch.arange(S, dtype=torch.int32).cuda(), sp.rope_freqs(pairs)[0]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_packed_and_in_place(inter, dtype):
    """Views of a packed [B, S, H + 2 Hk, D] on either side, in place, an odd offset, and q alone."""
    pos, freqs = _call_args()
    B, S, H, Hk, D = 2, 20, 4, 2, 64
    qkv = _rand((B, S, H + 2 * Hk, D), dtype, 5)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    want = sp.rope(q.contiguous(), k.contiguous(), pos, freqs, interleaved=inter)
    got = sp.rope(q, k, pos, freqs, interleaved=inter)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    alone, none = sp.rope(q, None, pos, freqs, interleaved=inter)
    assert torch.equal(alone, want[0]) and none is None
    out = torch.zeros_like(qkv)
    sp.rope(q, k, pos, freqs, interleaved=inter, q_out=out[:, :, :H].transpose(1, 2),
            k_out=out[:, :, H:H + Hk].transpose(1, 2))
    assert torch.equal(out[:, :, :H].transpose(1, 2), want[0])
    assert torch.equal(out[:, :, H:H + Hk].transpose(1, 2), want[1]) and int(out[:, :, H + Hk:].count_nonzero()) == 0
    odd = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(B, H, S, D)  # element-aligned only
    odd.copy_(q)
    assert torch.equal(sp.rope(odd, None, pos, freqs, interleaved=inter)[0], want[0])
    sp.rope(q, k, pos, freqs, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_expanded_input_and_transpose_property():
    """A broadcast input is read as it stands; rope_bwd is the transpose of rope (fp32, sums in fp64)."""
    pos, freqs = _call_args()
    x = _rand((1, 1, 20, 64), torch.float32, 7).expand(2, 3, 20, 64)
    y, _ = sp.rope(x, None, pos, freqs, mscale=1.1)
    assert torch.equal(y, sp.rope(x.contiguous(), None, pos, freqs, mscale=1.1)[0])
    w = _rand((2, 3, 20, 64), torch.float32, 8)
    g, _ = sp.rope_bwd(w, None, pos, freqs, mscale=1.1)
    a, b = (y.double() * w.double()).sum().item(), (x.double() * g.double()).sum().item()
    assert abs(a - b) <= 2.0 ** -19 * float((y.abs().double() * w.abs().double()).sum())


def test_stream_capture_and_empty():
    pos, freqs = _call_args()
    q = _rand((1, 2, 20, 64), torch.bfloat16, 9)
    want = sp.rope(q, q.clone(), pos, freqs)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sp.rope(q, None, pos, freqs, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, _ = sp.rope(q, None, pos, freqs)
    pos.add_(3)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, sp.rope(q, None, pos, freqs)[0]) and not torch.equal(y, want)
    e, _ = sp.rope(q[:, :, :0], None, pos[:0], freqs)
    assert e.shape == (1, 2, 0, 64)
    e, _ = sp.rope(q[:0], None, pos, freqs)
    assert e.shape == (0, 2, 20, 64)


def test_frequencies():
    f, m = sp.rope_freqs([3, 2], base=100.0)
    assert np.allclose(f.cpu(), [1, 100 ** (-1 / 3), 100 ** (-2 / 3), 1, 0.1]) and m == 1.0
    lin, _ = sp.rope_freqs(4, scaling="linear", factor=8.0)
    assert np.allclose(lin.cpu() * 8, sp.rope_freqs(4)[0].cpu())
    ntk, _ = sp.rope_freqs(4, scaling="ntk", factor=8.0)
    assert np.isclose(float(ntk[0]), 1.0) and np.isclose(float(ntk[3]) * 8, float(sp.rope_freqs(4)[0][3]))
    y, m = sp.rope_freqs(64, scaling="yarn", factor=8.0)
    base = sp.rope_freqs(64)[0].cpu()
    turns = 4096 * base / (2 * np.pi)
    assert np.allclose(y.cpu()[turns > 32], base[turns > 32]) and np.allclose(y.cpu()[turns < 1] * 8, base[turns < 1])
    assert np.isclose(m, 0.1 * np.log(8) + 1)


def test_refusals():
    pos, freqs = _call_args()
    q = _rand((1, 2, 20, 64), torch.bfloat16, 1)
    bad = [
        dict(q=q[0]), dict(q=q.cpu()), dict(q=q.double()), dict(q=q.transpose(2, 3)), dict(k=q.float()), dict(k=q[:, :, :5]),
        dict(pos=pos[:-1]), dict(pos=pos.long()), dict(pos=pos.cpu()), dict(freqs=freqs.float()), dict(freqs=freqs[:-1]),
        dict(rot_dim=63), dict(rot_dim=66), dict(rot_dim=-2), dict(sections=[16, 17]), dict(sections=[8, 8, 8, 8]),
        dict(sections=[40, -8]), dict(q_out=q[:, :, :10]), dict(q_out=q.float()), dict(k_out=q),
        dict(q_out=q[:, :1].expand(1, 2, 20, 64)),
    ]
    for over in bad:
        a = dict(q=q, k=None, pos=pos, freqs=freqs)
        kw = {n: v for n, v in over.items() if n not in a}
        a.update({n: v for n, v in over.items() if n in a})
        with pytest.raises(ValueError):
            sp.rope(a["q"], a["k"], a["pos"], a["freqs"], **kw)
    buf = _rand((1, 3, 20, 64), torch.bfloat16, 2)
    with pytest.raises(ValueError):  # shifted by a head: neither in place nor apart
        sp.rope(buf[:, :2], None, pos, freqs, q_out=buf[:, 1:])
    with pytest.raises(ValueError):
        sp.rope(buf[:, :1], buf[:, 1:2], pos, freqs, q_out=buf[:, 1:2])
    with pytest.raises(ValueError):
        out = torch.empty_like(q)
        sp.rope(q, q.clone(), pos, freqs, q_out=out, k_out=out)
