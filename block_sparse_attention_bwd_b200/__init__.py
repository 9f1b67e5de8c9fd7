"""Python binding of libspattn (exact block-sparse attention on B200).

Argument marshalling only: every step of the forward and backward passes
runs in the CUDA kernels of ``libspattn.so`` behind the C ABI declared in
``include/spattn.h``.  PyTorch supplies device memory and the current CUDA
stream.  There is no fallback: if the library is missing, importing this
package raises.

Calls launch on ``stream`` (by default the current one), and the tensors that
they make themselves come from that stream's memory pool: a program that reads
them on another stream orders the two and keeps the tensors until it has.

Names follow the C ABI: :class:`Plan` wraps ``spattn_plan``;
:func:`spattn_fwd`, :func:`spattn_bwd` and :func:`spattn_check` call the
entry points of the same names.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional, Tuple

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspattn.so")

SPATTN_OK = 0
SPATTN_ERR_INVALID_ARG, SPATTN_ERR_UNSUPPORTED, SPATTN_ERR_OOM, SPATTN_ERR_CUDA = 1, 2, 3, 4
SPATTN_ERR_TIMEOUT, SPATTN_ERR_DEVICE = 5, 6
STATUS_NAMES = {
    0: "SPATTN_OK",
    1: "SPATTN_ERR_INVALID_ARG",
    2: "SPATTN_ERR_UNSUPPORTED",
    3: "SPATTN_ERR_OOM",
    4: "SPATTN_ERR_CUDA",
    5: "SPATTN_ERR_TIMEOUT",
    6: "SPATTN_ERR_DEVICE",
}

ENTRY_POINTS = (
    "spattn_plan", "spattn_fwd", "spattn_bwd", "spattn_bwd_noalloc", "spattn_check", "spattn_plan_stats", "spattn_profile",
    "spattn_profile_read", "spattn_plan_pages", "spattn_plan_qblocks", "spattn_plan_work", "spattn_plan_destroy",
    "spattn_status_string", "spattn_wait_selftest", "spattn_plan_set_graph_device", "spattn_plan_entry_heads",
    "spattn_quantize_fp8", "spattn_fwd_fp8",
    "spattn_fwd_scored", "spattn_bwd_scored", "spattn_rope",
    "spattn_paged_create", "spattn_paged_destroy", "spattn_paged_workspace", "spattn_paged_fwd", "spattn_paged_check",
)


class SpattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({_lib().spattn_status_string(status).decode()})")


class _Layout(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("q_slots", ctypes.c_int64), ("kv_slots", ctypes.c_int64),
        ("q_group", ctypes.POINTER(ctypes.c_int32)), ("kv_group", ctypes.POINTER(ctypes.c_int32)),
        ("n_q_groups", ctypes.c_int32), ("n_kv_groups", ctypes.c_int32), ("scale", ctypes.c_float),
        ("kv_heads", ctypes.c_int32), ("graph_batches", ctypes.c_int32),
    ]


class _Score(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("k_pos", ctypes.c_void_p), ("q_last", ctypes.c_void_p), ("q_doc", ctypes.c_void_p),
                ("k_doc", ctypes.c_void_p), ("batches", ctypes.c_int32)]


class _RopeLayout(ctypes.Structure):
    # the stride arrays of spattn_rope_layout, element by element
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "batch", "heads", "kv_heads", "head_dim", "rot_dim",
                                              "interleaved", "inverse")] + [
        ("slots", ctypes.c_int64)] + [(f"{n}{i}", ctypes.c_int64) for n in ("q_stride", "k_stride", "q_out_stride",
                                                                           "k_out_stride") for i in range(3)] + [
        ("n_axes", ctypes.c_int32), ("section0", ctypes.c_int32), ("section1", ctypes.c_int32),
        ("section2", ctypes.c_int32), ("pos_batch_stride", ctypes.c_int64), ("mscale", ctypes.c_float)]


class _PagedLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("heads", "kv_heads", "head_dim", "page_slots", "max_seqs", "max_q",
                                              "max_kv")] + [("scale", ctypes.c_float), ("softcap", ctypes.c_float)]


class _PagedCall(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("tokens", ctypes.c_int64), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_slot_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
                ("v_slot_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("n_seqs", ctypes.c_int64),
                ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("slopes", ctypes.c_void_p),
                ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64)]


# The three structs as packed bytes, which a call builds in a fraction of the time
# that filling a ctypes structure takes.
_PACK_SCORE = struct.Struct("@f4x6Pi4x")
_PACK_ROPE = struct.Struct("@8i13q4iqf4x")
_PACK_PAGED = struct.Struct("@21q")
assert _PACK_SCORE.size == ctypes.sizeof(_Score) and _PACK_ROPE.size == ctypes.sizeof(_RopeLayout)
assert _PACK_PAGED.size == ctypes.sizeof(_PagedCall)


class _Graph(ctypes.Structure):
    _fields_ = [("row_ptr", ctypes.POINTER(ctypes.c_int64)), ("kv_groups", ctypes.POINTER(ctypes.c_int32))]


class _Stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "useful_pairs", "physical_pairs_fwd", "physical_pairs_dkdv", "physical_pairs_dq", "bsa_pairs",
        "n_work_fwd", "n_work_dkdv", "n_entries_fwd", "n_entries_dkdv", "device_bytes", "launches_fwd",
        "launches_bwd")] + [("plan_ms", ctypes.c_double)]


class _KernelTimes(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * 5), ("launches", ctypes.c_int64 * 5)]


KERNEL_NAMES = ("fwd", "fill", "delta", "dkdv", "dq")


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        I32, I64 = ctypes.c_int32, ctypes.c_int64
        lib.spattn_plan.argtypes = [ctypes.POINTER(_Layout), ctypes.POINTER(_Graph), ctypes.POINTER(P)]
        lib.spattn_fwd.argtypes = [P, P, P, P, P, P, P]
        lib.spattn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P]
        lib.spattn_fwd_scored.argtypes = [P, P, P, P, P, P, P, P]
        lib.spattn_bwd_scored.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P]
        lib.spattn_rope.argtypes = [P, P, P, P, P, P, P, P]
        lib.spattn_paged_create.argtypes = [ctypes.POINTER(_PagedLayout), ctypes.POINTER(P)]
        lib.spattn_paged_workspace.argtypes = [P, I64, ctypes.POINTER(I64)]
        lib.spattn_paged_fwd.argtypes = [P, P, P]
        lib.spattn_paged_check.argtypes = [P, P]
        lib.spattn_paged_destroy.argtypes = [P]
        lib.spattn_paged_destroy.restype = None
        lib.spattn_quantize_fp8.argtypes = [P, I64, I64, ctypes.c_int, P, P, P]
        lib.spattn_fwd_fp8.argtypes = [P, P, P, P, P, P, P, P, P]
        lib.spattn_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, P, P]
        lib.spattn_check.argtypes = [P, P]
        lib.spattn_wait_selftest.argtypes = [P, I64, P]
        lib.spattn_plan_set_graph_device.argtypes = [P, P, P, I64, P]
        lib.spattn_plan_stats.argtypes = [P, ctypes.POINTER(_Stats)]
        lib.spattn_plan_pages.argtypes = [P, I32, I64, ctypes.POINTER(ctypes.POINTER(I32)), ctypes.POINTER(I64)]
        lib.spattn_plan_qblocks.argtypes = [P, I32, I64, ctypes.POINTER(ctypes.POINTER(I32)), ctypes.POINTER(I64)]
        lib.spattn_plan_work.argtypes = [P, I32, ctypes.POINTER(ctypes.POINTER(I32)), ctypes.POINTER(I64),
                                         ctypes.POINTER(ctypes.POINTER(I32)), ctypes.POINTER(ctypes.POINTER(ctypes.c_uint64)),
                                         ctypes.POINTER(I64)]
        lib.spattn_plan_entry_heads.argtypes = [P, I32, ctypes.POINTER(ctypes.POINTER(ctypes.c_uint16)),
                                                ctypes.POINTER(I64)]
        lib.spattn_profile.argtypes = [P, ctypes.c_int]
        lib.spattn_profile_read.argtypes = [P, ctypes.POINTER(_KernelTimes)]
        lib.spattn_plan_destroy.argtypes = [P]
        lib.spattn_plan_destroy.restype = None
        lib.spattn_status_string.argtypes = [ctypes.c_int]
        lib.spattn_status_string.restype = ctypes.c_char_p
        for name in ENTRY_POINTS:
            if name not in ("spattn_plan_destroy", "spattn_paged_destroy", "spattn_status_string"):
                getattr(lib, name).restype = ctypes.c_int
        _LIB = lib
    return _LIB


def _check(status: int, where: str):
    if status != SPATTN_OK:
        raise SpattnError(status, where)


def _i32(a):
    return np.ascontiguousarray(a, dtype=np.int32)


class Plan:
    """Owning wrapper of ``spattn_plan_t``.

    ``q_group`` / ``kv_group``: int32 per slot (-1 = padded).  ``row_ptr`` /
    ``kv_groups``: CSR over (head, query group) of allowed key groups.
    The plan lives on the current CUDA device.
    """

    def __init__(self, q_group, kv_group, n_q_groups, n_kv_groups, row_ptr, kv_groups, *, batch, heads,
                 head_dim, scale=0.0, kv_heads=0, graph_batches=1):
        qg, kg = _i32(q_group), _i32(kv_group)
        rp = np.ascontiguousarray(row_ptr, dtype=np.int64)
        cols = _i32(kv_groups) if len(kv_groups) else np.zeros(1, np.int32)
        self._keep = (qg, kg, rp, cols)
        lay = _Layout(batch, heads, head_dim, qg.size, kg.size,
                      qg.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), kg.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                      int(n_q_groups), int(n_kv_groups), float(scale), int(kv_heads), int(graph_batches))
        gr = _Graph(rp.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), cols.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
        h = ctypes.c_void_p()
        _check(_lib().spattn_plan(ctypes.byref(lay), ctypes.byref(gr), ctypes.byref(h)), "spattn_plan")
        self.handle = h
        self.batch, self.heads, self.head_dim = batch, heads, head_dim
        self.kv_heads = heads if kv_heads == 0 else kv_heads
        self.q_slots, self.kv_slots = qg.size, kg.size
        self._keep = None

    @classmethod
    def from_problem(cls, problem, batch: Optional[int] = None):
        b = problem.batch if batch is None else batch
        gb = getattr(problem, "graph_batches", 1)
        if gb != 1 and b != problem.batch:
            raise ValueError("a problem with one graph per batch entry has a fixed batch")
        return cls(problem.q_group, problem.kv_group, problem.n_q_groups, problem.n_kv_groups, problem.row_ptr,
                   problem.kv_groups, batch=b, heads=problem.heads, head_dim=problem.head_dim, scale=problem.scale,
                   kv_heads=getattr(problem, "kv_heads", 0) or 0, graph_batches=gb)

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _lib().spattn_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_graph_device(self, row_ptr, kv_groups, stream=None):
        """Re-plan on the GPU for a new graph: ``row_ptr`` int64 and
        ``kv_groups`` int32, contiguous CUDA tensors in the spattn_graph
        format (spattn_plan_set_graph_device)."""
        import torch

        if row_ptr.dtype != torch.int64 or not row_ptr.is_cuda or not row_ptr.is_contiguous():
            raise ValueError("row_ptr: expected a contiguous CUDA int64 tensor")
        if kv_groups.dtype != torch.int32 or not kv_groups.is_cuda or not kv_groups.is_contiguous():
            raise ValueError("kv_groups: expected a contiguous CUDA int32 tensor")
        _check(_lib().spattn_plan_set_graph_device(self.handle, _ptr(row_ptr), _ptr(kv_groups), kv_groups.numel(),
                                                   _stream_handle(stream)), "spattn_plan_set_graph_device")

    def stats(self) -> dict:
        s = _Stats()
        _check(_lib().spattn_plan_stats(self.handle, ctypes.byref(s)), "spattn_plan_stats")
        return {n: getattr(s, n) for n, _ in _Stats._fields_}

    def profile(self, enable: bool):
        """Start / stop recording per-kernel CUDA events in fwd / bwd calls (clears the record)."""
        _check(_lib().spattn_profile(self.handle, 1 if enable else 0), "spattn_profile")

    def profile_read(self) -> dict:
        """{kernel: (summed ms, launches)} of the recorded launches; clears the record."""
        t = _KernelTimes()
        _check(_lib().spattn_profile_read(self.handle, ctypes.byref(t)), "spattn_profile_read")
        return {n: (t.ms[i], t.launches[i]) for i, n in enumerate(KERNEL_NAMES)}

    def pages(self, head: int, qblock: int) -> np.ndarray:
        ptr = ctypes.POINTER(ctypes.c_int32)()
        n = ctypes.c_int64()
        _check(_lib().spattn_plan_pages(self.handle, head, qblock, ctypes.byref(ptr), ctypes.byref(n)), "spattn_plan_pages")
        return np.ctypeslib.as_array(ptr, shape=(n.value,)).copy() if n.value else np.zeros(0, np.int32)

    def qblocks(self, head: int, page: int) -> np.ndarray:
        ptr = ctypes.POINTER(ctypes.c_int32)()
        n = ctypes.c_int64()
        _check(_lib().spattn_plan_qblocks(self.handle, head, page, ctypes.byref(ptr), ctypes.byref(n)), "spattn_plan_qblocks")
        return np.ctypeslib.as_array(ptr, shape=(n.value,)).copy() if n.value else np.zeros(0, np.int32)

    def entry_heads(self, which: int) -> np.ndarray:
        """Per entry of work list ``which``: its query head relative to the item's K/V head group."""
        return _entry_heads(self, which)

    def work(self, which: int) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
        """(work [n, 32] int32, pages [e] int32, masks [e, 2] uint64) of pass ``which`` (0 query-owned, 1
        key-owned); segment s of entry e is bits 16 (s % 4) of masks[e, s // 4]."""
        w = ctypes.POINTER(ctypes.c_int32)()
        p = ctypes.POINTER(ctypes.c_int32)()
        m = ctypes.POINTER(ctypes.c_uint64)()
        nw, ne = ctypes.c_int64(), ctypes.c_int64()
        _check(_lib().spattn_plan_work(self.handle, which, ctypes.byref(w), ctypes.byref(nw), ctypes.byref(p),
                                       ctypes.byref(m), ctypes.byref(ne)), "spattn_plan_work")
        work = np.ctypeslib.as_array(w, shape=(nw.value * 32,)).reshape(-1, 32).copy() if nw.value else np.zeros((0, 32), np.int32)
        pages = np.ctypeslib.as_array(p, shape=(ne.value,)).copy() if ne.value else np.zeros(0, np.int32)
        masks = (np.ctypeslib.as_array(m, shape=(2 * ne.value,)).reshape(-1, 2).copy() if ne.value
                 else np.zeros((0, 2), np.uint64))
        return work, pages, masks


def _entry_heads(plan, which):
    h = ctypes.POINTER(ctypes.c_uint16)()
    n = ctypes.c_int64()
    _check(_lib().spattn_plan_entry_heads(plan.handle, which, ctypes.byref(h), ctypes.byref(n)),
           "spattn_plan_entry_heads")
    return np.ctypeslib.as_array(h, shape=(n.value,)).copy() if n.value else np.zeros(0, np.uint16)


def _stream_handle(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_HERE = contextlib.nullcontext()


def _making_on(stream, t):
    """The context in which a call on ``stream`` makes its own tensors (results and workspaces), on the device of t.

    Memory from the current stream's pool may have just been freed there with its last kernels still
    running, and nothing orders those before a launch on another stream: the given stream's own pool it is.
    """
    torch = _torch()
    if stream is None or not isinstance(t, torch.Tensor) or not t.is_cuda:  # (no CUDA tensor: refused further on)
        return _HERE
    if stream.cuda_stream == _CURRENT_RAW_STREAM(t.device.index):
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=t.device)
    return torch.cuda.stream(stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape, dtype):
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or tuple(t.shape) != tuple(shape) \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")


def spattn_fwd(q, k, v, plan: Plan, o=None, lse=None, stream=None):
    """O [B,H,Sq,D] bf16 and LSE [B,H,Sq] fp32 for the plan's sparse graph."""
    import torch

    qs = (plan.batch, plan.heads, plan.q_slots, plan.head_dim)
    ks = (plan.batch, plan.kv_heads, plan.kv_slots, plan.head_dim)
    _need(q, "q", qs, torch.bfloat16)
    _need(k, "k", ks, torch.bfloat16)
    _need(v, "v", ks, torch.bfloat16)
    with _making_on(stream, q):
        if o is None:
            o = torch.empty(qs, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(qs[:3], dtype=torch.float32, device=q.device)
    _need(o, "o", qs, torch.bfloat16)
    _need(lse, "lse", qs[:3], torch.float32)
    _check(_lib().spattn_fwd(_ptr(q), _ptr(k), _ptr(v), plan.handle, _ptr(o), _ptr(lse), _stream_handle(stream)),
           "spattn_fwd")
    return o, lse


def quantize_fp8(x, stream=None):
    """E4M3 codes (uint8, same shape) and per-(batch, head) descale factors
    (float32 [B, H]) of a bf16 tensor [B, H, S, D], one slice per (batch, head)."""
    import torch

    if x.dim() != 4 or x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("quantize_fp8: x must be a contiguous CUDA bf16 tensor [B, H, S, D]")
    B, H, S, D = x.shape
    with _making_on(stream, x):
        x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
        descale = torch.empty((B, H), dtype=torch.float32, device=x.device)
    _check(_lib().spattn_quantize_fp8(_ptr(x), B * H, S, D, _ptr(x8), _ptr(descale), _stream_handle(stream)),
           "spattn_quantize_fp8")
    return x8, descale


def spattn_fwd_fp8(q8, k8, q_descale, k_descale, v, plan: Plan, o=None, lse=None, stream=None):
    """O and LSE of attention over the dequantised E4M3 Q and K (see quantize_fp8)."""
    import torch

    qs = (plan.batch, plan.heads, plan.q_slots, plan.head_dim)
    ks = (plan.batch, plan.kv_heads, plan.kv_slots, plan.head_dim)
    _need(q8, "q8", qs, torch.uint8)
    _need(k8, "k8", ks, torch.uint8)
    _need(v, "v", ks, torch.bfloat16)
    _need(q_descale, "q_descale", qs[:2], torch.float32)
    _need(k_descale, "k_descale", ks[:2], torch.float32)
    with _making_on(stream, q8):
        if o is None:
            o = torch.empty(qs, dtype=torch.bfloat16, device=q8.device)
        if lse is None:
            lse = torch.empty(qs[:3], dtype=torch.float32, device=q8.device)
    _need(o, "o", qs, torch.bfloat16)
    _need(lse, "lse", qs[:3], torch.float32)
    _check(_lib().spattn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(q_descale), _ptr(k_descale), _ptr(v), plan.handle, _ptr(o),
                                 _ptr(lse), _stream_handle(stream)), "spattn_fwd_fp8")
    return o, lse


def spattn_bwd(q, k, v, o, lse, do, plan: Plan, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV (bf16) given the forward's O and LSE and the loss gradient dO."""
    import torch

    qs = (plan.batch, plan.heads, plan.q_slots, plan.head_dim)
    ks = (plan.batch, plan.kv_heads, plan.kv_slots, plan.head_dim)
    for t, nm, sh in ((q, "q", qs), (k, "k", ks), (v, "v", ks), (o, "o", qs), (do, "do", qs)):
        _need(t, nm, sh, torch.bfloat16)
    _need(lse, "lse", qs[:3], torch.float32)
    with _making_on(stream, q):
        dq = torch.empty(qs, dtype=torch.bfloat16, device=q.device) if dq is None else dq
        dk = torch.empty(ks, dtype=torch.bfloat16, device=q.device) if dk is None else dk
        dv = torch.empty(ks, dtype=torch.bfloat16, device=q.device) if dv is None else dv
    _need(dq, "dq", qs, torch.bfloat16)
    _need(dk, "dk", ks, torch.bfloat16)
    _need(dv, "dv", ks, torch.bfloat16)
    _check(_lib().spattn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), plan.handle, _ptr(dq), _ptr(dk),
                             _ptr(dv), _stream_handle(stream)), "spattn_bwd")
    return dq, dk, dv


class Score:
    """Score modification of :func:`spattn_fwd_scored` / :func:`spattn_bwd_scored` (``spattn_score``).

    ``softcap`` c > 0 caps scores as ``c tanh(x / c)`` (0: none); ``slopes``
    (fp32 [heads]) subtracts ``slopes[h] |q_pos - k_pos|``; ``q_last`` allows only
    keys with ``k_pos <= q_last`` (``q_pos`` itself for a causal mask,
    ``maximum(q_pos, prefix - 1)`` for one with a prefix); ``q_doc`` / ``k_doc``
    allow only keys of the query's own document (negative ids attend nothing).
    ``q_*`` are int32 CUDA tensors [q_slots] or [batch, q_slots], ``k_*`` the same
    over kv_slots, all contiguous and all with or all without the batch dimension.
    """

    def __init__(self, softcap=0.0, slopes=None, q_pos=None, k_pos=None, q_last=None, q_doc=None, k_doc=None):
        self.softcap = float(softcap)
        self.slopes, self.q_pos, self.k_pos, self.q_last, self.q_doc, self.k_doc = slopes, q_pos, k_pos, q_last, q_doc, k_doc

    def _packed(self, plan: Plan, device) -> bytes:
        torch = _torch()
        i32 = torch.int32
        ptrs, dims, slopes = [], 0, self.slopes
        if slopes is not None:
            _want(slopes, "slopes", (plan.heads,), torch.float32, device)
            slopes = slopes.data_ptr()
        nq, nk = plan.q_slots, plan.kv_slots
        for t, name, slots in ((self.q_pos, "q_pos", nq), (self.k_pos, "k_pos", nk), (self.q_last, "q_last", nq),
                               (self.q_doc, "q_doc", nq), (self.k_doc, "k_doc", nk)):
            if t is None:
                ptrs.append(0)
                continue
            batched = isinstance(t, torch.Tensor) and t.dim() == 2
            _want(t, name, (plan.batch, slots) if batched else (slots,), i32, device)
            dims |= 2 if batched else 1
            ptrs.append(t.data_ptr())
        if dims == 3:
            raise ValueError("score arrays: either all or none have a batch dimension")
        return _PACK_SCORE.pack(self.softcap, slopes or 0, *ptrs, plan.batch if dims == 2 else 1)


_TORCH = None
_CURRENT_RAW_STREAM = None


def _torch():
    global _TORCH, _CURRENT_RAW_STREAM
    if _TORCH is None:
        import torch

        # (without the Stream object around the handle, where torch offers that)
        _CURRENT_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream",
                                      lambda index: torch.cuda.current_stream(index).cuda_stream)
        _TORCH = torch
    return _TORCH


def _want(t, name, shape, dtype, device):
    """_need, and on the given device (a CUDA one)."""
    if not isinstance(t, _TORCH.Tensor) or t.dtype is not dtype or t.device != device or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)} on {device}")


def _raw_stream(stream, device):
    """The stream's handle; without one, that of the current stream of ``device``."""
    if stream is not None:
        return stream.cuda_stream
    return _CURRENT_RAW_STREAM(device.index)


def _device_of(t, name):
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, not {type(t).__name__}")
    return t.device


def _current_device_of(t, name):
    """The tensor's device, which a call with a plan needs to be the current one (the plan's is checked there)."""
    dev = _device_of(t, name)
    if dev.index != _torch().cuda.current_device():
        raise ValueError(f"{name}: is on {dev}, but the current device is cuda:{_torch().cuda.current_device()}")
    return dev


def spattn_fwd_scored(q, k, v, plan: Plan, score: Score, o=None, lse=None, stream=None):
    """O [B,H,Sq,D] bf16 and LSE [B,H,Sq] fp32 for the plan's sparse graph with modified scores."""
    torch = _torch()
    dev, bf16 = _current_device_of(q, "q"), torch.bfloat16
    qs = (plan.batch, plan.heads, plan.q_slots, plan.head_dim)
    ks = (plan.batch, plan.kv_heads, plan.kv_slots, plan.head_dim)
    _want(q, "q", qs, bf16, dev)
    _want(k, "k", ks, bf16, dev)
    _want(v, "v", ks, bf16, dev)
    sc = score._packed(plan, dev)
    with _making_on(stream, q):
        if o is None:
            o = torch.empty_like(q)
        else:
            _want(o, "o", qs, bf16, dev)
        if lse is None:
            lse = q.new_empty(qs[:3], dtype=torch.float32)
        else:
            _want(lse, "lse", qs[:3], torch.float32, dev)
    _check(_lib().spattn_fwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), plan.handle, sc,
                                    o.data_ptr(), lse.data_ptr(), _raw_stream(stream, dev)), "spattn_fwd_scored")
    return o, lse


def spattn_bwd_scored(q, k, v, o, lse, do, plan: Plan, score: Score, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV (bf16) of :func:`spattn_fwd_scored` with the same score, given its O and LSE and the loss gradient dO."""
    torch = _torch()
    dev, bf16 = _current_device_of(q, "q"), torch.bfloat16
    qs = (plan.batch, plan.heads, plan.q_slots, plan.head_dim)
    ks = (plan.batch, plan.kv_heads, plan.kv_slots, plan.head_dim)
    _want(q, "q", qs, bf16, dev)
    _want(k, "k", ks, bf16, dev)
    _want(v, "v", ks, bf16, dev)
    _want(o, "o", qs, bf16, dev)
    _want(do, "do", qs, bf16, dev)
    _want(lse, "lse", qs[:3], torch.float32, dev)
    sc = score._packed(plan, dev)
    with _making_on(stream, q):
        if dq is None:
            dq = torch.empty_like(q)
        else:
            _want(dq, "dq", qs, bf16, dev)
        if dk is None:
            dk = torch.empty_like(k)
        else:
            _want(dk, "dk", ks, bf16, dev)
        if dv is None:
            dv = torch.empty_like(k)
        else:
            _want(dv, "dv", ks, bf16, dev)
    _check(_lib().spattn_bwd_scored(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                    do.data_ptr(), plan.handle, sc, dq.data_ptr(), dk.data_ptr(),
                                    dv.data_ptr(), _raw_stream(stream, dev)), "spattn_bwd_scored")
    return dq, dk, dv


def rope_freqs(sections, base=10000.0, scaling=None, factor=1.0, original_slots=4096, beta_fast=32.0, beta_slow=1.0,
               device="cuda"):
    """(freqs, mscale) for :func:`rope`: fp64 radians per position of every pair.

    ``sections``: pairs per position axis (an int for one axis); each axis has its
    own ladder ``base ** (-i / n)``.  ``scaling`` for contexts ``factor`` times the
    trained one: ``None``; ``"linear"`` divides every frequency by the factor;
    ``"ntk"`` raises the base by ``factor ** (n / (n - 1))``, so that the slowest
    pair is divided by the factor and the fastest kept; ``"yarn"`` divides pairs
    that make fewer than ``beta_slow`` turns over ``original_slots`` positions, keeps
    those above ``beta_fast`` turns, blends between (linearly in the turns, as the
    method's paper has it; where a checkpoint ramps linearly in the pair's index
    instead, pass its own ``freqs`` to :func:`rope`), and sets mscale = 0.1 ln(factor) + 1.
    """
    import math

    import torch

    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"rope_freqs: unknown scaling {scaling!r}")
    if not (base > 0 and factor > 0):
        raise ValueError("rope_freqs: base and factor must be positive")
    if scaling == "yarn" and not (original_slots > 0 and beta_fast > beta_slow):
        raise ValueError("rope_freqs: original_slots must be positive and beta_fast above beta_slow")
    sections = [int(sections)] if isinstance(sections, (int, np.integer)) else [int(n) for n in sections]
    if any(n < 0 for n in sections):
        raise ValueError("rope_freqs: sections must not be negative")
    ladders, mscale = [], 1.0
    for n in sections:
        i = np.arange(n, dtype=np.float64)
        b = base * factor ** (n / (n - 1)) if scaling == "ntk" and n > 1 else base
        f = float(b) ** (-i / n) if n else i
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            turns = original_slots * f / (2 * math.pi)
            keep = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0.0, 1.0)
            f = f * keep + f / factor * (1 - keep)
            mscale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        ladders.append(f)
    return torch.from_numpy(np.concatenate(ladders) if ladders else np.zeros(0)).to(device), mscale


def _rope_rows(t, what, name, dtype, device):
    """Shape and strides of a [B, H, S, D] tensor of a rope call, checked."""
    if not isinstance(t, _TORCH.Tensor) or t.dtype is not dtype or t.device != device or t.dim() != 4:
        raise ValueError(f"{name}: {what} must be a {dtype} tensor [B, H, S, D] on {device}, as q is")
    shape, stride = t.shape, t.stride()
    if stride[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name}: {what} must be contiguous in its last dimension")
    return shape, stride


def _rope_out(t, shape):
    """A contiguous tensor like t, and its strides."""
    y = _TORCH.empty_like(t) if t.is_contiguous() else t.new_empty(tuple(shape))
    return y, y.stride()


def _sums_reach(terms, lo, hi):
    """Whether some sum of k_i stride_i, k_i from first_i to last_i, lies in [lo, hi].

    ``terms``: (stride, first, last), those of one stride added up.  With the largest strides first, few k_i of each leave a sum that the
    smaller ones can still bring there, wherever strides nest as a tensor's do.  True without an
    answer after some thousand of them.
    """
    ranges = {}
    for st, first, last in terms:
        if st:
            a, b = ranges.get(st, (0, 0))
            ranges[st] = (a + first, b + last)
    terms = [(st, *ranges[st]) for st in sorted(ranges, reverse=True)]
    least, most = [0], [0]  # of the sums of the last terms
    for st, first, last in reversed(terms):
        least.append(least[-1] + st * first)
        most.append(most[-1] + st * last)
    left = 4000

    def search(i, lo, hi):
        nonlocal left
        if i == len(terms):
            return lo <= 0 <= hi
        st, first, last = terms[i]
        rest = len(terms) - 1 - i
        for k in range(max(first, -((most[rest] - lo) // st)), min(last, (hi - least[rest]) // st) + 1):
            left -= 1
            if left < 0 or search(i + 1, lo - k * st, hi - k * st):
                return True
        return False

    return search(0, lo, hi)


def _view_repeats(shape, stride):
    """Whether two elements of a [B, H, S, D] view share an address."""
    (b, h, n, d), (x, y, z, _) = shape, stride
    e, f = (n - 1) * z + d, (h - 1) * y + d  # what the rows of a head span, and those of a slot
    if (n == 1 or z >= d) and (h == 1 or y >= e) and (b == 1 or x >= e + f - d):
        return False  # every stride passes over what the smaller ones reach, heads in order ...
    if (h == 1 or y >= d) and (n == 1 or z >= f) and (b == 1 or x >= e + f - d):
        return False  # ... or slots
    dims = sorted(((st, m) for st, m in ((x, b), (y, h), (z, n)) if m > 1), reverse=True)
    return any(_sums_reach([(dims[i][0], 1, dims[i][1] - 1)] + [(st, 1 - n, n - 1) for st, n in dims[i + 1:]], 1 - d, d - 1)
               for i in range(len(dims)))


def _views_meet(x, y, size):
    """Whether two [B, H, S, D] views (address, shape, strides) share an address."""
    (at, (bx, hx, sx, d), (b0, h0, s0, _)), (to, (by, hy, sy, _), (b1, h1, s1, _)) = x, y
    gap = (to - at) // size
    # Parts of one packed buffer: both repeat with one period, in which they lie apart (slots of a
    # [B, S, heads, D] one, rows of a [B, H, S, 2 D] one).
    if s0 == s1 and b0 == b1 and s0 > 0 and b0 % s0 == 0:
        if h0 % s0 == 0 and h1 % s0 == 0:
            if d <= gap % s0 <= s0 - d:
                return False
        elif (hx - 1) * h0 + d <= gap % s0 <= s0 - (hy - 1) * h1 - d:
            return False
    return _sums_reach([(b0, 0, bx - 1), (h0, 0, hx - 1), (s0, 0, sx - 1), (b1, 1 - by, 0), (h1, 1 - hy, 0), (s1, 1 - sy, 0)],
                       gap + 1 - d, gap + d - 1)


def _rope_overlaps(name, ins, outs, size):
    """Refuses outputs that share an address with each other or, without being in place of it, with an input.

    ``ins``, ``outs``: (address, shape, strides) of the [B, H, S, D] tensors; ``size``: bytes of an element.
    """
    spans = []  # [first, end) byte addresses that the rows touch
    for at, (b, h, n, d), (x, y, z, _) in ins + outs:
        spans.append((at, at + ((b - 1) * x + (h - 1) * y + (n - 1) * z + d) * size))
    n = len(ins)
    for _, shape, stride in outs:
        if _view_repeats(shape, stride):
            raise ValueError(f"{name}: an output has elements that share an address")
    if n == 2 and spans[2][0] < spans[3][1] and spans[3][0] < spans[2][1] and _views_meet(outs[0], outs[1], size):
        raise ValueError(f"{name}: the two outputs share an address")
    for i in range(n):
        first, end = spans[n + i]
        for j in range(n):
            if first >= spans[j][1] or spans[j][0] >= end:
                continue
            x, y = ins[j], outs[i]
            if i == j and y[0] == x[0] and all(a == b or m == 1 for a, b, m in zip(x[2], y[2], x[1])):
                continue  # in place: an element is read and written by one thread
            if _views_meet(y, x, size):
                raise ValueError(f"{name}: an output overlaps an input without being in place of it")


def _rope(name, inverse, q, k, pos, freqs, rot_dim, interleaved, sections, mscale, q_out, k_out, stream):
    torch = _torch()
    dev, dt = _device_of(q, name), q.dtype
    code = 0 if dt is torch.bfloat16 else 1 if dt is torch.float16 else 2 if dt is torch.float32 else None
    if code is None:
        raise ValueError(f"{name}: q must be bf16, fp16 or fp32")
    qs, a = _rope_rows(q, "q", name, dt, dev)
    B, H, S, D = qs
    Hk, ks, b = 0, None, a
    if k is not None:
        ks, b = _rope_rows(k, "k", name, dt, dev)
        Hk = ks[1]
        if Hk < 1 or ks[0] != B or ks[2] != S or ks[3] != D:
            raise ValueError(f"{name}: k must have shape {(B, 'heads', S, D)}")
    elif k_out is not None:
        raise ValueError(f"{name}: an output for k without k")
    if H < 1 or D < 1:
        raise ValueError(f"{name}: q must have at least one head and one element per row")
    rot = D if rot_dim is None else int(rot_dim)
    if rot < 0 or rot > D or rot % 2:
        raise ValueError(f"{name}: rot_dim must be even and between 0 and {D}")
    pairs = rot // 2
    sec = (pairs,) if sections is None else tuple(map(int, sections))
    axes = len(sec)
    if not 1 <= axes <= 3 or min(sec) < 0 or sum(sec) != pairs:
        raise ValueError(f"{name}: sections must be one to three counts that sum to rot_dim / 2 = {pairs}")
    if not isinstance(pos, torch.Tensor) or pos.dtype is not torch.int32 or pos.device != dev \
            or not pos.is_contiguous() or not (pos.shape == (axes, S) or pos.shape == (B, axes, S)
                                               or (axes == 1 and pos.shape == (S,))):
        raise ValueError(f"{name}: pos must be a contiguous int32 tensor {(axes, S)} or {(B, axes, S)}"
                         + (f" or {(S,)}" if axes == 1 else "") + f" on {dev}")
    _want(freqs, "freqs", (pairs,), torch.float64, dev)
    given = q_out is not None or k_out is not None
    with _making_on(stream, q):
        if q_out is None:
            q_out, c = _rope_out(q, qs)
        else:
            shape, c = _rope_rows(q_out, "the output for q", name, dt, dev)
            if shape != qs:
                raise ValueError(f"{name}: the output for q must have shape {tuple(qs)}")
        d = c
        if Hk:
            if k_out is None:
                k_out, d = _rope_out(k, ks)
            else:
                shape, d = _rope_rows(k_out, "the output for k", name, dt, dev)
                if shape != ks:
                    raise ValueError(f"{name}: the output for k must have shape {tuple(ks)}")
    q_at, o_at = q.data_ptr(), q_out.data_ptr()
    k_at, p_at = (k.data_ptr(), k_out.data_ptr()) if Hk else (None, None)
    if given and B and S:
        _rope_overlaps(name, [(q_at, qs, a), (k_at, ks, b)] if Hk else [(q_at, qs, a)],
                       [(o_at, qs, c), (p_at, ks, d)] if Hk else [(o_at, qs, c)], 4 if code == 2 else 2)
    lay = _PACK_ROPE.pack(code, B, H, Hk, D, rot, 1 if interleaved else 0, 1 if inverse else 0, S, a[0], a[1], a[2],
                          b[0], b[1], b[2], c[0], c[1], c[2], d[0], d[1], d[2], axes, sec[0],
                          sec[1] if axes > 1 else 0, sec[2] if axes > 2 else 0, axes * S if pos.dim() == 3 else 0,
                          mscale)
    args = (lay, q_at, k_at, pos.data_ptr(), freqs.data_ptr(), o_at, p_at, _raw_stream(stream, dev))
    if torch.cuda.current_device() == dev.index:
        status = _lib().spattn_rope(*args)
    else:
        with torch.cuda.device(dev):
            status = _lib().spattn_rope(*args)
    _check(status, "spattn_rope")
    return q_out, k_out


def rope(q, k, pos, freqs, *, rot_dim=None, interleaved=False, sections=None, mscale=1.0, q_out=None, k_out=None,
         stream=None):
    """Rotary positions of Q [B,H,S,D] and K [B,Hk,S,D] (or None) in one launch; returns both.

    Inputs and outputs may be strided views (bf16, fp16 or fp32; the last dimension
    contiguous), an output may be its input, and views of one buffer are told
    apart by their addresses; new outputs are contiguous, as spattn_fwd wants them.  ``pos``: int32 [S], [axes, S] or [B, axes, S];
    ``sections``: pairs per position axis (one axis by default); ``freqs``, ``mscale``:
    see :func:`rope_freqs`.  ``interleaved`` pairs elements 2p and 2p + 1, else p
    and p + rot_dim / 2; elements from ``rot_dim`` on are copied.
    """
    return _rope("rope", False, q, k, pos, freqs, rot_dim, interleaved, sections, mscale, q_out, k_out, stream)


def rope_bwd(dq_out, dk_out, pos, freqs, *, rot_dim=None, interleaved=False, sections=None, mscale=1.0, dq=None,
             dk=None, stream=None):
    """Gradient of :func:`rope`: dQ and dK of its inputs from those of its outputs (same arguments)."""
    return _rope("rope_bwd", True, dq_out, dk_out, pos, freqs, rot_dim, interleaved, sections, mscale, dq, dk, stream)


class PagedPlan:
    """Owning wrapper of ``spattn_paged_t``: the bounds of paged attention calls.

    ``page_slots``: slots per page (a multiple of 16); ``max_seqs``, ``max_q`` (new
    tokens of one sequence; 1 for decoding) and ``max_kv`` (cache slots of one
    sequence) bound every call; ``softcap`` and ``slopes`` (fp32 [heads] on the GPU)
    modify the scores as in :class:`Score`.  Lives on the current CUDA device.
    """

    def __init__(self, *, heads, kv_heads, head_dim, page_slots, max_seqs, max_q, max_kv, scale=0.0, softcap=0.0,
                 slopes=None):
        import torch

        lay = _PagedLayout(heads, kv_heads, head_dim, page_slots, max_seqs, max_q, max_kv, float(scale), float(softcap))
        h = ctypes.c_void_p()
        _check(_lib().spattn_paged_create(ctypes.byref(lay), ctypes.byref(h)), "spattn_paged_create")
        self.handle = h
        self.heads, self.kv_heads, self.head_dim, self.page_slots = heads, kv_heads, head_dim, page_slots
        self.max_seqs, self.max_q, self.max_kv = max_seqs, max_q, max_kv
        if slopes is not None:
            _need(slopes, "slopes", (heads,), torch.float32)
        self.slopes = slopes
        self._bytes = {}

    def workspace_bytes(self, n_seqs: int) -> int:
        """Bytes of workspace of a call with ``n_seqs`` sequences."""
        if n_seqs not in self._bytes:
            n = ctypes.c_int64()
            _check(_lib().spattn_paged_workspace(self.handle, n_seqs, ctypes.byref(n)), "spattn_paged_workspace")
            self._bytes[n_seqs] = n.value
        return self._bytes[n_seqs]

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _lib().spattn_paged_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def spattn_paged_fwd(q, k_cache, v_cache, page_table, q_start, kv_len, paged: PagedPlan, o=None, lse=None,
                     workspace=None, stream=None):
    """Attention of each sequence's new tokens over a paged cache; returns O [T, H, D] bf16 and LSE [T, H] fp32.

    ``q`` [T, H, D] bf16 (token and head strides free); ``k_cache`` / ``v_cache``
    [pages, page_slots, kv_heads, D] bf16, or a permuted view of [kv_heads, slots, D];
    ``page_table`` int32 [n, P]; ``q_start`` int32 [n + 1]; ``kv_len`` int32 [n], the new
    tokens included.  Rows of o and lse that no sequence names are left as they are
    (undefined in the tensors that the call makes itself).  ``workspace``: a uint8
    CUDA tensor of ``paged.workspace_bytes(n)`` bytes; by default the call allocates one.
    """
    torch = _torch()
    H, Hk, D, ps = paged.heads, paged.kv_heads, paged.head_dim, paged.page_slots
    dev, bf16, i32 = _current_device_of(q, "q"), torch.bfloat16, torch.int32
    if q.dtype is not bf16 or q.dim() != 3 or q.shape[1:] != (H, D) or q.stride(2) != 1:
        raise ValueError(f"q: expected a CUDA bf16 tensor [tokens, {H}, {D}], contiguous in its last dimension")
    T = q.shape[0]
    pages = k_cache.shape[0] if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 4 else -1
    strides = []
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(t, torch.Tensor) or t.device != dev or t.dtype is not bf16 or t.shape != (pages, ps, Hk, D) \
                or t.stride(3) != 1:
            raise ValueError(f"{name}: expected a bf16 tensor [pages, {ps}, {Hk}, {D}] on {dev}, contiguous in its "
                             "last dimension")
        st = t.stride()
        if pages > 1 and st[0] != ps * st[1]:
            raise ValueError(f"{name}: pages must follow each other (page stride = {ps} slot strides)")
        strides += [st[1], st[2] if Hk > 1 else 0]
    if not isinstance(kv_len, torch.Tensor) or kv_len.dim() != 1:
        raise ValueError("kv_len: expected an int32 tensor [sequences]")
    n = kv_len.shape[0]
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError(f"page_table: expected an int32 tensor [{n}, pages]")
    width = page_table.shape[1]
    _want(page_table, "page_table", (n, width), i32, dev)
    _want(q_start, "q_start", (n + 1,), i32, dev)
    _want(kv_len, "kv_len", (n,), i32, dev)
    slopes = paged.slopes
    if slopes is not None:
        _want(slopes, "slopes", (H,), torch.float32, dev)
    need = paged.workspace_bytes(n)
    with _making_on(stream, q):
        if o is None:
            o = q.new_empty((T, H, D))
        else:
            _want(o, "o", (T, H, D), bf16, dev)
        if lse is None:
            lse = q.new_empty((T, H), dtype=torch.float32)
        else:
            _want(lse, "lse", (T, H), torch.float32, dev)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None and (not isinstance(workspace, torch.Tensor) or workspace.device != dev
                                  or workspace.dtype is not torch.uint8 or not workspace.is_contiguous()):
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {dev}")
    # (the stride of a single token or head means nothing)
    c = _PACK_PAGED.pack(q.data_ptr(), q.stride(0) if T > 1 else 0, q.stride(1) if H > 1 else 0, T,
                         k_cache.data_ptr(), v_cache.data_ptr(), *strides, pages, page_table.data_ptr(), width, n, q_start.data_ptr(), kv_len.data_ptr(),
                         0 if slopes is None else slopes.data_ptr(), o.data_ptr(), lse.data_ptr(),
                         0 if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel())
    _check(_lib().spattn_paged_fwd(paged.handle, c, _raw_stream(stream, dev)), "spattn_paged_fwd")
    return o, lse


def spattn_paged_check(paged: PagedPlan, stream=None):
    """Synchronise the stream and raise if a paged call recorded a device-side error."""
    _check(_lib().spattn_paged_check(paged.handle, _stream_handle(stream)), "spattn_paged_check")


def spattn_check(plan: Plan, stream=None):
    """Synchronise the stream and raise if a kernel recorded a device-side error."""
    _check(_lib().spattn_check(plan.handle, _stream_handle(stream)), "spattn_check")


def spattn_wait_selftest(plan: Plan, deadline_cycles: int, stream=None) -> int:
    """Run the bounded-wait failure self-test; returns the following spattn_check status."""
    _check(_lib().spattn_wait_selftest(plan.handle, int(deadline_cycles), _stream_handle(stream)),
           "spattn_wait_selftest")
    return _lib().spattn_check(plan.handle, _stream_handle(stream))


def load_library():
    """Load libspattn.so (raises ImportError when it has not been built)."""
    return _lib()
