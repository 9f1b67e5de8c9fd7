"""Scored attention, rotary positions and paged attention, float64, by definition.

Test infrastructure only (see the package docstring); nothing here is shared
with the CUDA path.  Besides each value there is a bound on how far an
implementation that keeps everything in fp32 but rounds weights, dS and
outputs to bf16 may be from it, element by element:

* a rounding to bf16 is off by at most 2^-8 of the value (half a unit of eps =
  2^-7), so O = sum P v with rounded weights and a rounded result is off by at
  most 2^-8 (sum P |v| + |O|);
* Delta = sum_d dO O, formed from the rounded O, inherits that bound times |dO|
  (rows in ``exact_delta`` have it from their weights: fp32's part only);
* dS = P f (dP - Delta) (f = 1 - tanh^2) is off by P f of Delta's bound and by
  its own rounding, dV's weights by theirs;
* fp32 adds sums of D products, the score and exp, covered by ``_FP32`` of the
  absolute sums they run over.  A score that is off by e changes its weight by
  a factor 1 + e; scores here are below 2^6 in size, so e < 2^-24 * 2^6 * 8 =
  2^-15 with the products' own summation included;
* f below fp32's normal numbers (2^-126) cannot be told from up to four of them.
"""

from __future__ import annotations

import numpy as np

_BF16 = 2.0 ** -8
_FP32 = 2.0 ** -14
_F_FLOOR = 2.0 ** -123


def scores(q, k, scale, softcap=0.0, slope=0.0, q_pos=None, k_pos=None):
    """(z, f): modified scores and d z / d (scale q.k)."""
    x = scale * (q @ k.T)
    f = np.ones_like(x)
    if softcap > 0:
        u = x / softcap
        # 1 - tanh^2 as 1 / cosh^2: the difference would lose everything beyond |u| = 18
        x, f = softcap * np.tanh(u), 1.0 / np.cosh(np.clip(u, -350.0, 350.0)) ** 2
    if slope != 0.0:
        x = x - slope * np.abs(np.asarray(q_pos, np.float64)[:, None] - np.asarray(k_pos, np.float64)[None, :])
    return x, f


def score_mask(mask, k_pos=None, q_last=None, q_doc=None, k_doc=None):
    """The graph's token mask narrowed by positions and documents."""
    m = np.array(mask, dtype=bool)
    if q_last is not None:
        m &= np.asarray(k_pos, np.int64)[None, :] <= np.asarray(q_last, np.int64)[:, None]
    if q_doc is not None:
        m &= (np.asarray(q_doc)[:, None] == np.asarray(k_doc)[None, :]) & (np.asarray(q_doc) >= 0)[:, None]
    return m


def softmax(z, mask):
    """(P, LSE) with P = 0 and LSE = -inf on empty rows."""
    some = mask.any(axis=1)
    zm = np.where(mask, z, -np.inf)
    top = np.where(some, zm.max(axis=1, initial=-np.inf), 0.0)
    e = np.where(mask, np.exp(np.where(mask, z, 0.0) - top[:, None]), 0.0)
    l = np.where(some, e.sum(axis=1), 1.0)
    return e / l[:, None], np.where(some, top + np.log(l), -np.inf)


def forward(q, k, v, mask, z):
    """O, LSE and their bounds."""
    p, lse = softmax(z, mask)
    o = p @ v
    spread = p @ np.abs(v)
    o_tol = _BF16 * (spread + np.abs(o)) * (1 + _BF16) + _FP32 * spread
    lse_tol = np.where(np.isfinite(lse), 2.0 ** -15 + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse), lse, 0.0)), 0.0)
    return o, lse, o_tol, lse_tol


def backward(q, k, v, do, mask, z, f, scale, exact_delta=None):
    """{name: (value, bound)} of dq, dk, dv of one head."""
    p, _ = softmax(z, mask)
    o = p @ v
    o_tol = _BF16 * (p @ np.abs(v) + np.abs(o)) * (1 + _BF16)
    dp = do @ v.T
    adp = np.abs(do) @ np.abs(v).T
    delta = (p * dp).sum(axis=1, keepdims=True)
    delta_tol = (np.abs(do) * o_tol).sum(axis=1, keepdims=True)
    if exact_delta is not None:
        delta_tol = np.where(np.asarray(exact_delta)[:, None], 0.0, delta_tol)
    ds = p * f * (dp - delta)
    mass = adp + (p * adp).sum(axis=1, keepdims=True)
    fuzz = p * f * (delta_tol + _FP32 * mass) + _F_FLOOR * p * mass
    ds_tol = fuzz + _BF16 * (np.abs(ds) + fuzz)
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    spread = np.abs(p).T @ np.abs(do)

    def done(x, tol, mass):
        return x, tol + _BF16 * (np.abs(x) + tol) + _FP32 * mass

    return {"dq": done(dq, scale * ds_tol @ np.abs(k), scale * np.abs(ds) @ np.abs(k)),
            "dk": done(dk, scale * ds_tol.T @ np.abs(q), scale * np.abs(ds).T @ np.abs(q)),
            "dv": done(dv, _BF16 * spread, spread)}


def rope(x, pos, freqs, sections, rot_dim, interleaved, mscale=1.0, inverse=False):
    """Rotary positions of x [..., S, D]; pos [axes, S] integers, freqs [rot_dim / 2]."""
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = np.asarray(pos, np.float64)[axis].T * np.asarray(freqs, np.float64)
    c, s = mscale * np.cos(ang), mscale * np.sin(ang) * (-1.0 if inverse else 1.0)
    y = np.array(x, np.float64)
    i = np.arange(rot_dim // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
    a, b = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    return y


def paged(q, k_rows, v_rows, kv_len, scale, softcap=0.0, slopes=None):
    """O [n, H, D], LSE [n, H] and bounds of one sequence's n new tokens over its kv_len cached
    rows ([kv_len, kv_heads, D], in order); query head h reads K/V head h * kv_heads // H."""
    n, H, D = q.shape
    kv_heads = k_rows.shape[1]
    q_pos, k_pos = np.arange(kv_len - n, kv_len), np.arange(kv_len)
    mask = k_pos[None, :] <= q_pos[:, None]
    out = [np.zeros((n, H, D)), np.zeros((n, H)), np.zeros((n, H, D)), np.zeros((n, H))]
    for h in range(H):
        hk = h * kv_heads // H
        z, _ = scores(q[:, h], k_rows[:, hk], scale, softcap, 0.0 if slopes is None else float(slopes[h]), q_pos, k_pos)
        r = forward(q[:, h], k_rows[:, hk], v_rows[:, hk], mask, z)
        for dst, x in zip(out, r):
            dst[:, h] = x
    return out
