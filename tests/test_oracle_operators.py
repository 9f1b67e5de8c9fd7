"""The fp64 oracle of the scored, rotary and paged operators against
something other than itself: torch autograd, central differences, complex
multiplication and closed forms."""

import numpy as np
import pytest
import torch

from oracle import operators as R


def _case(seed, n=13, m=17, d=8):
    rng = np.random.default_rng(seed)
    q, k, v, do = (rng.standard_normal(s) for s in ((n, d), (m, d), (m, d), (n, d)))
    mask = rng.random((n, m)) < 0.8
    mask[3] = False
    return rng, q, k, v, do, mask


@pytest.mark.parametrize("cap,slope", [(0.0, 0.0), (1.5, 0.0), (0.0, 0.3), (2.0, 0.2)])
def test_scored_matches_autograd_and_differences(cap, slope):
    rng, q, k, v, do, mask = _case(1)
    qp, kp = rng.integers(-5, 30, 13), rng.integers(-5, 30, 17)
    scale = 0.4

    def loss_parts(q, k, v):
        z, f = R.scores(q, k, scale, cap, slope, qp, kp)
        return z, f

    z, f = loss_parts(q, k, v)
    o, lse, _, _ = R.forward(q, k, v, mask, z)
    g = R.backward(q, k, v, do, mask, z, f, scale)
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v)]
    x = scale * t[0] @ t[1].T
    if cap:
        x = cap * torch.tanh(x / cap)
    x = x - slope * torch.tensor(np.abs(qp[:, None] - kp[None, :]).astype(float))
    x = x.masked_fill(~torch.tensor(mask), -1e30)
    w = torch.softmax(x, dim=1) * torch.tensor(mask.any(1, keepdims=True))
    ot = w @ t[2]
    (ot * torch.tensor(do)).sum().backward()
    assert np.allclose(ot.detach().numpy(), o, atol=1e-12)
    assert np.allclose(torch.logsumexp(x, 1).detach().numpy()[mask.any(1)], lse[mask.any(1)], atol=1e-12)
    assert (o[3] == 0).all() and lse[3] == -np.inf and (g["dq"][0][3] == 0).all()
    for name, a in zip(("dq", "dk", "dv"), t):
        assert np.allclose(a.grad.numpy(), g[name][0], atol=1e-11), name
    # central differences of the loss along random directions
    h = 1e-5
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        d = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
        d[i] = rng.standard_normal(d[i].shape)

        def loss(s):
            a = [q + s * d[0], k + s * d[1], v + s * d[2]]
            return float((R.forward(a[0], a[1], a[2], mask, loss_parts(*a)[0])[0] * do).sum())

        num = (loss(h) - loss(-h)) / (2 * h)
        assert abs(num - float((g[name][0] * d[i]).sum())) <= 1e-6 * max(1.0, abs(num)), name


def test_score_mask_by_hand():
    m = R.score_mask(np.ones((3, 4), bool), k_pos=[0, 1, 2, 3], q_last=[0, 2, -1], q_doc=[5, 5, 5], k_doc=[5, 7, 5, 5])
    assert m.tolist() == [[True, False, False, False], [True, False, True, False], [False] * 4]
    m = R.score_mask(np.ones((2, 2), bool), q_doc=[-1, 0], k_doc=[-1, 0])
    assert m.tolist() == [[False, False], [False, True]]


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_is_complex_multiplication_and_orthogonal(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 5, 10))
    pos = np.array([[0, 3, -7, 100, 9], [1, 1, 2, 2, 50]])
    freqs = np.array([1.0, 0.1, 0.01])
    y = R.rope(x, pos, freqs, [2, 1], 6, interleaved, mscale=1.25)
    pair = (lambda a: (a[..., 0:6:2], a[..., 1:6:2])) if interleaved else (lambda a: (a[..., :3], a[..., 3:6]))
    ang = np.stack([pos[0] * 1.0, pos[0] * 0.1, pos[1] * 0.01], axis=1)
    want = (pair(x)[0] + 1j * pair(x)[1]) * 1.25 * np.exp(1j * ang)
    assert np.allclose(pair(y)[0] + 1j * pair(y)[1], want, atol=1e-12)
    assert (y[..., 6:] == x[..., 6:]).all()
    back = R.rope(y, pos, freqs, [2, 1], 6, interleaved, mscale=1 / 1.25, inverse=True)
    assert np.allclose(back, x, atol=1e-12)
    # the inverse is the transpose: <rope(x), w> = <x, rope_inverse(w)> (both scaled by mscale)
    w = rng.standard_normal(x.shape)
    assert abs((y * w).sum() - (x * R.rope(w, pos, freqs, [2, 1], 6, interleaved, 1.25, inverse=True)).sum()) < 1e-10


def test_paged_is_causal_attention_of_the_last_rows():
    rng = np.random.default_rng(3)
    k, v, q = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 4, 4))
    full = R.paged(q, k, v, 9, 0.5, 3.0, [0.1, 0.2, 0.3, 0.0])
    part = R.paged(q[6:], k, v, 9, 0.5, 3.0, [0.1, 0.2, 0.3, 0.0])
    for a, b in zip(full, part):
        assert np.allclose(a[6:], b)
    # the first token sees its own key only
    assert np.allclose(full[0][0], v[0, [0, 0, 1, 1]])
