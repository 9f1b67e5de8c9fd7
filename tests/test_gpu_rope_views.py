"""Rope calls with outputs among the views of one packed buffer."""

import pytest
import torch

import block_sparse_attention_bwd_b200 as sp

pytestmark = pytest.mark.gpu

B, S, H, HK, D = 2, 333, 4, 2, 64


def _inputs():
    gen = torch.Generator().manual_seed(3)
    qkv = torch.randn((B, S, H + 2 * HK, D), generator=gen).bfloat16().cuda()
    pos, (freqs, _) = torch.arange(S, dtype=torch.int32).cuda(), sp.rope_freqs(D // 2)
    view = lambda t, a, b: t[:, :, a:b].transpose(1, 2)  # noqa: E731
    want = sp.rope(view(qkv, 0, H).contiguous(), view(qkv, H, H + HK).contiguous(), pos, freqs)
    return qkv, view, pos, freqs, want


@pytest.mark.parametrize("which", ["q", "k", "both"])
def test_one_of_two_in_place(which):
    qkv, view, pos, freqs, want = _inputs()
    kept = qkv.clone()
    q, k = view(qkv, 0, H), view(qkv, H, H + HK)
    got = sp.rope(q, k, pos, freqs, q_out=None if which == "k" else q, k_out=None if which == "q" else k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if which == "q":
        assert torch.equal(k, view(kept, H, H + HK))
    if which == "k":
        assert torch.equal(q, view(kept, 0, H))
    assert torch.equal(qkv[:, :, H + HK:], kept[:, :, H + HK:])


def test_into_unused_heads_of_the_same_buffer():
    qkv, view, pos, freqs, want = _inputs()
    wide = torch.cat([qkv, torch.zeros_like(qkv)], 2)
    n = H + 2 * HK
    sp.rope(view(wide, 0, H), view(wide, H, H + HK), pos, freqs, q_out=view(wide, n, n + H), k_out=view(wide, n + H, n + H + HK))
    assert torch.equal(view(wide, n, n + H), want[0]) and torch.equal(view(wide, n + H, n + H + HK), want[1])
    assert torch.equal(wide[:, :, :n], qkv) and int(wide[:, :, n + H + HK:].count_nonzero()) == 0


def test_outputs_that_share_heads_are_refused():
    qkv, view, pos, freqs, _ = _inputs()
    out = torch.zeros_like(qkv)
    for a, b in ((view(out, 0, H), view(out, 2, 2 + HK)), (view(out, 3, 3 + H), view(out, 6, 6 + HK))):
        with pytest.raises(ValueError):
            sp.rope(view(qkv, 0, H), view(qkv, H, H + HK), pos, freqs, q_out=a, k_out=b)
    assert int(out.count_nonzero()) == 0
