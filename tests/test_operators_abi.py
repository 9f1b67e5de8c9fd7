"""Refusals of the scored, rotary and paged entry points that need no GPU:
the status codes of the C ABI for bad arguments, before anything is launched."""

import ctypes

import numpy as np
import pytest

import block_sparse_attention_bwd_b200 as sp
from workloads import configs as W

INVALID, UNSUPPORTED = sp.SPATTN_ERR_INVALID_ARG, sp.SPATTN_ERR_UNSUPPORTED
OKPTR = 1 << 20  # an aligned address that no rejected call may touch


def _plan():
    return sp.Plan.from_problem(W.make_problem("tiny"))


def _fwd(plan, score, q=OKPTR):
    return sp.load_library().spattn_fwd_scored(q, OKPTR, OKPTR, plan.handle, score, OKPTR, OKPTR, None)


def test_score_arguments():
    plan = _plan()
    lib = sp.load_library()
    good = dict(softcap=0.0, batches=1)
    bad = [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(batches=0), dict(batches=2),
           dict(slopes=OKPTR), dict(slopes=OKPTR, q_pos=OKPTR), dict(q_last=OKPTR), dict(q_doc=OKPTR), dict(k_doc=OKPTR),
           dict(q_last=OKPTR + 2, k_pos=OKPTR), dict(q_doc=OKPTR, k_doc=OKPTR + 1)]
    for b in bad:
        assert _fwd(plan, ctypes.byref(sp._Score(**{**good, **b}))) == INVALID, b
        assert lib.spattn_bwd_scored(OKPTR, OKPTR, OKPTR, OKPTR, OKPTR, OKPTR, plan.handle,
                                     ctypes.byref(sp._Score(**{**good, **b})), OKPTR, OKPTR, OKPTR, None) == INVALID, b
    assert _fwd(plan, None) == INVALID
    assert lib.spattn_fwd_scored(OKPTR, OKPTR, OKPTR, None, ctypes.byref(sp._Score(**good)), OKPTR, OKPTR, None) == INVALID
    plan.close()


def _rope(over=None, **ptr):
    f = dict(dtype=0, batch=1, heads=2, kv_heads=1, head_dim=64, rot_dim=32, interleaved=0, inverse=0, slots=4, n_axes=1,
             section0=16, section1=0, section2=0, pos_batch_stride=0, mscale=1.0)
    f.update(over or {})
    p = dict(q=OKPTR, k=OKPTR, pos=OKPTR, freqs=OKPTR, qo=OKPTR, ko=OKPTR)
    p.update(ptr)
    return sp.load_library().spattn_rope(ctypes.byref(sp._RopeLayout(**f)), p["q"], p["k"], p["pos"], p["freqs"], p["qo"],
                                         p["ko"], None)


def test_rope_arguments():
    for o in (dict(dtype=3), dict(dtype=-1), dict(batch=-1), dict(heads=0), dict(kv_heads=-1), dict(head_dim=0),
              dict(rot_dim=33), dict(rot_dim=66), dict(rot_dim=-2), dict(n_axes=0), dict(n_axes=4), dict(section0=15),
              dict(n_axes=2, section0=20, section1=-4), dict(mscale=float("nan")), dict(slots=-1)):
        assert _rope(o) == INVALID, o
    assert _rope(dict(head_dim=1025)) == UNSUPPORTED and _rope(dict(heads=40000)) == UNSUPPORTED
    for p in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(freqs=None),
              dict(q=OKPTR + 1), dict(freqs=OKPTR + 4), dict(pos=OKPTR + 2)):
        assert _rope(**p) == INVALID, p
    assert _rope(dict(dtype=2), q=OKPTR + 2) == INVALID
    assert sp.load_library().spattn_rope(None, OKPTR, None, OKPTR, OKPTR, OKPTR, None, None) == INVALID
    # nothing to do: no pointer is looked at
    assert _rope(dict(slots=0), q=None) == 0 and _rope(dict(batch=0), q=None) == 0


def _paged(**over):
    a = dict(heads=8, kv_heads=2, head_dim=128, page_slots=16, max_seqs=4, max_q=16, max_kv=4096)
    a.update(over)
    return sp.PagedPlan(**a)


@pytest.mark.parametrize("over,code", [
    (dict(heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(kv_heads=0), INVALID), (dict(page_slots=8), INVALID),
    (dict(page_slots=24), INVALID), (dict(max_seqs=0), INVALID), (dict(max_q=0), INVALID), (dict(max_kv=0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(softcap=-0.5), INVALID),
    (dict(softcap=float("inf")), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(max_seqs=70000), UNSUPPORTED),
    (dict(max_kv=(1 << 30) + 1), UNSUPPORTED), (dict(max_q=1 << 28), UNSUPPORTED),
])
def test_paged_layouts(over, code):
    with pytest.raises(sp.SpattnError) as e:
        _paged(**over)
    assert e.value.status == code


def test_paged_workspace_is_bounded_and_grows_with_nothing_else():
    p = _paged()
    assert p.workspace_bytes(0) == 0 and p.workspace_bytes(1) >= 0
    with pytest.raises(sp.SpattnError):
        p.workspace_bytes(5)
    # partial rows (head_dim + 4 fp32 each) of split tiles: sixteen rounds of two CTAs per SM at most
    for kw in (dict(max_q=4096, max_kv=1 << 20), dict(max_seqs=512, max_kv=1 << 17), dict(max_q=1, max_kv=1 << 24),
               dict(max_seqs=65535, max_kv=1 << 20, max_q=1)):
        q = _paged(**kw)
        rows = kw.get("max_q", 16) * 4
        for n in (1, q.max_seqs):
            tiles = n * 2 * -(-rows // 128)
            assert q.workspace_bytes(n) <= max(tiles, 16 * 2 * 160) * min(rows, 128) * 132 * 4
        q.close()
    p.close()


def test_paged_call_arguments():
    lib = sp.load_library()
    p = _paged()
    good = dict(q=OKPTR, q_token_stride=1024, q_head_stride=128, tokens=4, k_cache=OKPTR, v_cache=OKPTR, k_slot_stride=256,
                k_head_stride=128, v_slot_stride=256, v_head_stride=128, n_pages=10, page_table=OKPTR, table_stride=8,
                n_seqs=2, q_start=OKPTR, kv_len=OKPTR, o=OKPTR, lse=OKPTR, workspace=OKPTR, workspace_bytes=1 << 40)

    def status(**over):
        return lib.spattn_paged_fwd(p.handle, ctypes.byref(sp._PagedCall(**{**good, **over})), None)

    for o in (dict(q=None), dict(q=OKPTR + 8), dict(k_cache=None), dict(v_cache=OKPTR + 4), dict(o=None), dict(page_table=None),
              dict(q_start=OKPTR + 2), dict(kv_len=None), dict(lse=OKPTR + 2), dict(slopes=OKPTR + 1), dict(q_token_stride=4),
              dict(q_head_stride=-8), dict(k_slot_stride=120), dict(v_slot_stride=100), dict(k_head_stride=64),
              dict(n_seqs=5), dict(n_seqs=-1), dict(tokens=-1), dict(n_pages=0), dict(n_pages=-1), dict(table_stride=0)):
        assert status(**o) == INVALID, o
    for o in (dict(n_pages=1 << 40), dict(tokens=1 << 32), dict(table_stride=1 << 33)):
        assert status(**o) == UNSUPPORTED, o
    assert status(n_seqs=0, q=None) == 0 and status(tokens=0, q=None) == 0
    assert lib.spattn_paged_fwd(None, ctypes.byref(sp._PagedCall(**good)), None) == INVALID
    assert lib.spattn_paged_fwd(p.handle, None, None) == INVALID
    assert lib.spattn_paged_workspace(None, 1, None) == INVALID and lib.spattn_paged_check(None, None) == INVALID
    lib.spattn_paged_destroy(None)
    p.close()


def test_binding_refuses_cpu_tensors():
    import torch

    x = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sp.rope(x, None, torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    plan = _plan()
    with pytest.raises(ValueError):
        sp.spattn_fwd_scored(x, x, x, plan, sp.Score(softcap=1.0))
    with pytest.raises(ValueError):
        sp.spattn_bwd_scored(x, x, x, x, x, x, plan, sp.Score(softcap=1.0))
    p = _paged()
    with pytest.raises(ValueError):
        sp.spattn_paged_fwd(x[0], x, x, None, None, None, p)
    assert np.isclose(sp.rope_freqs(4, device="cpu")[0][1].item(), 10000 ** -0.25)
    for bad in (dict(scaling="cubic"), dict(factor=0.0), dict(base=-1.0)):
        with pytest.raises(ValueError):
            sp.rope_freqs(4, device="cpu", **bad)
    with pytest.raises(ValueError):
        sp.rope_freqs([4, -1], device="cpu")
    p.close()
    plan.close()
