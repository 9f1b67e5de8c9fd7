"""Frequencies of rotary positions, on the CPU: the ramp of "yarn", and arguments without one."""

import numpy as np
import pytest

import block_sparse_attention_bwd_b200 as sp


def test_yarn_blends_linearly_in_the_turns():
    base = sp.rope_freqs(64, device="cpu")[0].numpy()
    f, m = sp.rope_freqs(64, scaling="yarn", factor=8.0, original_slots=2048, beta_fast=20.0, beta_slow=2.0, device="cpu")
    turns = 2048 * base / (2 * np.pi)
    part = (turns > 2) & (turns < 20)
    assert part.sum() > 5
    keep = (turns[part] - 2) / 18
    assert np.allclose(f.numpy()[part], base[part] * (keep + (1 - keep) / 8), rtol=1e-12)
    assert np.allclose(f.numpy()[turns >= 20], base[turns >= 20]) and np.allclose(f.numpy()[turns <= 2] * 8, base[turns <= 2])
    assert np.isclose(m, 0.1 * np.log(8) + 1)


@pytest.mark.parametrize("over", [dict(beta_fast=2.0, beta_slow=2.0), dict(beta_fast=1.0, beta_slow=4.0),
                                  dict(original_slots=0), dict(beta_fast=float("nan"))])
def test_yarn_without_a_ramp_is_refused(over):
    """(equal ends of the ramp gave NaN frequencies, exchanged ones kept the slow pairs and divided the fast)"""
    with pytest.raises(ValueError):
        sp.rope_freqs(64, scaling="yarn", factor=8.0, device="cpu", **over)
    f, _ = sp.rope_freqs(64, device="cpu", **over)  # not looked at without it
    assert np.isfinite(f.numpy()).all()
