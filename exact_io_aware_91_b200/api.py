"""Python binding of the C ABI in ``include/fa.h`` (argument marshalling only).

Every function here has the name of the C entry point it calls.  PyTorch provides
device memory and the current CUDA stream; all arithmetic happens in the CUDA
kernels of ``libfa_b200.so``.  There is no fallback: if the library is missing
or the device is not supported, the call raises.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

from . import build as _build

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5
FA_ERR_RANGE = 6
FA_ERR_INDEX = 7
FA_ERR_NO_PAGES = 8

FA_BF16 = 0
FA_F16 = 1

EXPORTS = ("fa_fwd", "fa_fwd_gqa", "fa_fwd_workspace_size", "fa_fwd_ws", "fa_fwd_f32", "fa_bwd_workspace_size", "fa_bwd", "fa_bwd_gqa_workspace_size",
           "fa_bwd_gqa", "fa_bwd_ws_workspace_size", "fa_bwd_ws", "fa_attn_fwd_workspace_size", "fa_attn_fwd", "fa_attn_bwd_workspace_size", "fa_attn_bwd",
           "fa_attn_fwd_fp8_workspace_size", "fa_attn_fwd_fp8", "fa_bwd_noalloc", "fa_last_device_status",
           "fa_paged_attn_workspace_size", "fa_paged_attn", "fa_pages_write", "fa_pages_workspace_size", "fa_pages_copy",
           "fa_pages_reserve", "fa_pages_fork", "fa_pages_free", "fa_pages_compact",
           "fa_device_status", "fa_bwd_set_phase_events", "fa_selftest_wait_timeout", "fa_selftest_paged_give_up", "fa_selftest_exp2",
           "fa_status_str")

# Size of the scratch array fa_bwd_noalloc uses instead of a caller workspace.
FA_BWD_NOALLOC_MAX_WORKSPACE = 64 << 20


class FaAttnProblem(ctypes.Structure):
    """``fa_attn_problem`` of ``include/fa.h``."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("H_kv", ctypes.c_int), ("N", ctypes.c_int),
                ("d", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("window_left", ctypes.c_int), ("window_right", ctypes.c_int)]


class FaPagedProblem(ctypes.Structure):
    """``fa_paged_problem`` of ``include/fa.h``."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("H_kv", ctypes.c_int), ("T", ctypes.c_int),
                ("d", ctypes.c_int), ("dtype", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("max_pages", ctypes.c_int), ("table_stride", ctypes.c_int),
                ("prefix_len", ctypes.c_int), ("causal", ctypes.c_int), ("scale", ctypes.c_float),
                ("k_stride", ctypes.c_longlong * 3), ("v_stride", ctypes.c_longlong * 3)]


class FaPageTable(ctypes.Structure):
    """``fa_page_table`` of ``include/fa.h``."""
    _fields_ = [("rows", ctypes.c_int), ("max_pages", ctypes.c_int), ("table_stride", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int), ("block_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("ref_counts", ctypes.c_void_p)]


class FaPagePlanes(ctypes.Structure):
    """``fa_page_planes`` of ``include/fa.h``."""
    _fields_ = [("planes", ctypes.POINTER(ctypes.c_void_p)), ("n_planes", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_bytes", ctypes.c_longlong), ("page_stride", ctypes.c_longlong)]


class FAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {status_str(status)} ({status})")
        self.status = status


_LIB = None


def library() -> ctypes.CDLL:
    """Load ``libfa_b200.so`` from the package directory (raises if it is not built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m exact_io_aware_91_b200.build` "
            "(there is no non-CUDA fallback)"
        )
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_gqa.restype = i
    lib.fa_fwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_fwd_workspace_size.restype = sz
    lib.fa_fwd_ws.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_fwd_ws.restype = i
    lib.fa_fwd_f32.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_f32.restype = i
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_gqa_workspace_size.argtypes = [i, i, i, i, i]
    lib.fa_bwd_gqa_workspace_size.restype = sz
    lib.fa_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp]
    lib.fa_bwd_gqa.restype = i
    lib.fa_bwd_ws_workspace_size.argtypes = [i, i, i, i, i]
    lib.fa_bwd_ws_workspace_size.restype = sz
    lib.fa_bwd_ws.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, sz, vp, sz, vp]
    lib.fa_bwd_ws.restype = i
    pp = ctypes.POINTER(FaAttnProblem)
    lib.fa_attn_fwd_workspace_size.argtypes = [pp]
    lib.fa_attn_fwd_workspace_size.restype = sz
    lib.fa_attn_fwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fa_attn_fwd.restype = i
    lib.fa_attn_bwd_workspace_size.argtypes = [pp]
    lib.fa_attn_bwd_workspace_size.restype = sz
    lib.fa_attn_bwd.argtypes = [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fa_attn_bwd.restype = i
    lib.fa_attn_fwd_fp8_workspace_size.argtypes = [pp]
    lib.fa_attn_fwd_fp8_workspace_size.restype = sz
    lib.fa_attn_fwd_fp8.argtypes = [pp, vp, vp, vp, f, f, f, vp, vp, vp, sz, vp]
    lib.fa_attn_fwd_fp8.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_bwd_noalloc.restype = i
    pg = pt = pl = vp  # fa_paged_problem, fa_page_table, fa_page_planes: a byref() or packed bytes
    lib.fa_paged_attn_workspace_size.argtypes = [pg]
    lib.fa_paged_attn_workspace_size.restype = sz
    lib.fa_paged_attn.argtypes = [pg, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fa_paged_attn.restype = i
    lib.fa_pages_write.argtypes = [pg, vp, vp, vp, vp, vp, vp, vp]
    lib.fa_pages_write.restype = i
    lib.fa_pages_workspace_size.argtypes = [i, i]
    lib.fa_pages_workspace_size.restype = sz
    lib.fa_pages_copy.argtypes = [pl, vp, vp, i, vp]
    lib.fa_pages_copy.restype = i
    lib.fa_pages_reserve.argtypes = [pt, vp, vp, sz, vp]
    lib.fa_pages_reserve.restype = i
    lib.fa_pages_fork.argtypes = [pl, pt, vp, vp, i, vp, sz, vp]
    lib.fa_pages_fork.restype = i
    lib.fa_pages_free.argtypes = [pt, vp, i, vp]
    lib.fa_pages_free.restype = i
    lib.fa_pages_compact.argtypes = [pl, pt, vp, vp, vp, vp, sz, vp]
    lib.fa_pages_compact.restype = i
    lib.fa_selftest_paged_give_up.argtypes = [pg, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, vp]
    lib.fa_selftest_paged_give_up.restype = i
    lib.fa_selftest_wait_timeout.argtypes = [vp]
    lib.fa_selftest_wait_timeout.restype = i
    lib.fa_selftest_exp2.argtypes = [vp, vp, i, vp]
    lib.fa_selftest_exp2.restype = i
    lib.fa_last_device_status.argtypes = [vp]
    lib.fa_last_device_status.restype = i
    lib.fa_device_status.argtypes = [vp]
    lib.fa_device_status.restype = i
    lib.fa_bwd_set_phase_events.argtypes = [vp]
    lib.fa_bwd_set_phase_events.restype = None
    lib.fa_status_str.argtypes = [i]
    lib.fa_status_str.restype = ctypes.c_char_p
    _LIB = lib
    return lib


def status_str(status: int) -> str:
    return library().fa_status_str(int(status)).decode()


fa_status_str = status_str


def _stream_handle(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(fn: str, status: int) -> None:
    if status != FA_OK:
        raise FAError(fn, status)


def _shape(q: torch.Tensor) -> tuple[int, int, int, int]:
    if q.dim() != 4:
        raise ValueError("expected a (B, H, N, d) tensor")
    return tuple(int(x) for x in q.shape)  # type: ignore[return-value]


def _same(*ts: torch.Tensor, dtype: torch.dtype, shape) -> None:
    for t in ts:
        if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"expected contiguous CUDA {dtype} tensors of shape {tuple(shape)}")


def _scale(scale, d: int) -> float:
    return float(1.0 / math.sqrt(d) if scale is None else scale)


def fa_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False, scale: float | None = None,
           o: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention forward on bf16 (B, H, N, d) CUDA tensors (C ``fa_fwd``).  Returns (o, lse).

    The residual a training forward can hand to the backward is written by ``fa_fwd_gqa``,
    ``fa_fwd_ws`` and ``fa_attn_fwd`` (``save_residual=True``)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, dtype=torch.bfloat16, shape=(B, H, N, d))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _same(o, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    st = library().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                          _scale(scale, d), int(bool(causal)), _stream_handle(stream))
    _check("fa_fwd", st)
    return o, lse


def _gqa_heads(q: torch.Tensor, k: torch.Tensor) -> int:
    if k.dim() != 4 or k.shape[0] != q.shape[0] or k.shape[2:] != q.shape[2:]:
        raise ValueError("k, v must be (B, H_kv, N, d) with q's B, N and d")
    h_kv = int(k.shape[1])
    if h_kv < 1 or q.shape[1] % h_kv:
        raise ValueError("the query head count must be a multiple of the key/value head count")
    return h_kv


def fa_fwd_gqa(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
               scale: float | None = None, o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               o_resid: torch.Tensor | None = None, save_residual: bool = False, stream=None):
    """Grouped-query / multi-query forward: q (B, H, N, d), k and v (B, H_kv, N, d) bf16.

    Query head h reads key/value head h // (H // H_kv).  Returns like ``fa_fwd``."""
    B, H, N, d = _shape(q)
    H_kv = _gqa_heads(q, k)
    _same(q, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(k, v, dtype=torch.bfloat16, shape=(B, H_kv, N, d))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if o_resid is None and save_residual:
        o_resid = torch.empty_like(q)
    _same(o, dtype=torch.bfloat16, shape=(B, H, N, d))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    st = library().fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                              None if o_resid is None else o_resid.data_ptr(), B, H, H_kv, N, d, _scale(scale, d),
                              int(bool(causal)), _stream_handle(stream))
    _check("fa_fwd_gqa", st)
    return (o, lse) if o_resid is None else (o, lse, o_resid)


def fa_fwd_workspace_size(B: int, H_kv: int, N: int, d: int) -> int:
    return int(library().fa_fwd_workspace_size(B, H_kv, N, d))


def fa_fwd_ws(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
              scale: float | None = None, o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
              o_resid: torch.Tensor | None = None, save_residual: bool = False, workspace=None, stream=None):
    """Forward with a workspace (V converted to fp16 in one pass before the kernel); k, v may
    have fewer heads than q (grouped-query).  Returns like ``fa_fwd``."""
    B, H, N, d = _shape(q)
    H_kv = _gqa_heads(q, k)
    _same(q, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(k, v, dtype=torch.bfloat16, shape=(B, H_kv, N, d))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if o_resid is None and save_residual:
        o_resid = torch.empty_like(q)
    _same(o, dtype=torch.bfloat16, shape=(B, H, N, d))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    if workspace is None:
        workspace = torch.empty(max(fa_fwd_workspace_size(B, H_kv, N, d), 1), dtype=torch.uint8, device=q.device)
    st = library().fa_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                             None if o_resid is None else o_resid.data_ptr(), B, H, H_kv, N, d, _scale(scale, d),
                             int(bool(causal)), workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    _check("fa_fwd_ws", st)
    return (o, lse) if o_resid is None else (o, lse, o_resid)


def fa_fwd_f32(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
               scale: float | None = None, stream=None):
    """fp32 forward (no input rounding). Returns (o, lse)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, dtype=torch.float32, shape=(B, H, N, d))
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    st = library().fa_fwd_f32(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                              _scale(scale, d), int(bool(causal)), _stream_handle(stream))
    _check("fa_fwd_f32", st)
    return o, lse


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(library().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None, workspace=None,
           dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV (fp32) of sum(O * dO) (C ``fa_bwd``; rowsum(dO * O) from the bf16 O --
    ``fa_bwd_gqa`` / ``fa_attn_bwd`` take the forward's residual).  Returns (dq, dk, dv)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, do, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    if dq is None:
        dq = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty_like(dq)
    if dv is None:
        dv = torch.empty_like(dq)
    _same(dq, dk, dv, dtype=torch.float32, shape=(B, H, N, d))
    ws_bytes = fa_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    if workspace.numel() < ws_bytes:  # the C call trusts the size (its signature carries none)
        raise ValueError(f"workspace of {workspace.numel()} bytes, fa_bwd needs {ws_bytes}")
    st = library().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, _scale(scale, d),
                          int(bool(causal)), workspace.data_ptr(), _stream_handle(stream))
    _check("fa_bwd", st)
    return dq, dk, dv


def fa_bwd_gqa_workspace_size(B: int, H: int, H_kv: int, N: int, d: int) -> int:
    return int(library().fa_bwd_gqa_workspace_size(B, H, H_kv, N, d))


def fa_bwd_gqa(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None, workspace=None,
               dq=None, dk=None, dv=None, o_resid=None, stream=None):
    """Grouped-query backward: dq (B, H, N, d); dk, dv (B, H_kv, N, d), summed over each group."""
    B, H, N, d = _shape(q)
    H_kv = _gqa_heads(q, k)
    _same(q, o, do, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(k, v, dtype=torch.bfloat16, shape=(B, H_kv, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    if dq is None:
        dq = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty((B, H_kv, N, d), dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty_like(dk)
    _same(dq, dtype=torch.float32, shape=(B, H, N, d))
    _same(dk, dv, dtype=torch.float32, shape=(B, H_kv, N, d))
    ws_bytes = fa_bwd_gqa_workspace_size(B, H, H_kv, N, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
    st = library().fa_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              None if o_resid is None else o_resid.data_ptr(), do.data_ptr(), lse.data_ptr(),
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, H_kv, N, d, _scale(scale, d),
                              int(bool(causal)), workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    _check("fa_bwd_gqa", st)
    return dq, dk, dv


def fa_bwd_ws_workspace_size(B: int, H: int, H_kv: int, N: int, d: int) -> int:
    return int(library().fa_bwd_ws_workspace_size(B, H, H_kv, N, d))


def fa_bwd_ws(q, k, v, o, do, lse, fwd_workspace, causal: bool = False, scale: float | None = None,
              workspace=None, dq=None, dk=None, dv=None, o_resid=None, stream=None):
    """``fa_bwd_gqa`` that takes the fp16 V copy from ``fwd_workspace``, the workspace of the
    ``fa_fwd_ws`` call that produced o (and lse, o_resid) from this v.  Returns (dq, dk, dv)."""
    B, H, N, d = _shape(q)
    H_kv = _gqa_heads(q, k)
    _same(q, o, do, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(k, v, dtype=torch.bfloat16, shape=(B, H_kv, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    if fwd_workspace is None or fwd_workspace.device != q.device:
        raise ValueError("fa_bwd_ws needs the forward's workspace on the inputs' device")
    if dq is None:
        dq = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty((B, H_kv, N, d), dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty_like(dk)
    _same(dq, dtype=torch.float32, shape=(B, H, N, d))
    _same(dk, dv, dtype=torch.float32, shape=(B, H_kv, N, d))
    if workspace is None:
        workspace = torch.empty(max(fa_bwd_ws_workspace_size(B, H, H_kv, N, d), 1), dtype=torch.uint8,
                                device=q.device)
    st = library().fa_bwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             None if o_resid is None else o_resid.data_ptr(), do.data_ptr(), lse.data_ptr(),
                             dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, H_kv, N, d, _scale(scale, d),
                             int(bool(causal)), fwd_workspace.data_ptr(), fwd_workspace.numel(),
                             workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    _check("fa_bwd_ws", st)
    return dq, dk, dv


def _problem(q, k, causal, scale, window) -> FaAttnProblem:
    B, H, N, d = _shape(q)
    H_kv = _gqa_heads(q, k)
    wl, wr = window
    return FaAttnProblem(B, H, H_kv, N, d, _scale(scale, d), int(bool(causal)), int(wl), int(wr))


def fa_attn_fwd_workspace_size(problem: FaAttnProblem) -> int:
    return int(library().fa_attn_fwd_workspace_size(ctypes.byref(problem)))


def fa_attn_bwd_workspace_size(problem: FaAttnProblem) -> int:
    return int(library().fa_attn_bwd_workspace_size(ctypes.byref(problem)))


def fa_attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, window=(-1, -1), o=None, lse=None,
                o_resid=None, save_residual: bool = False, workspace=None, stream=None):
    """Forward with every option: grouped K/V heads (k, v (B, H_kv, N, d)) and a sliding
    window (left, right) (-1 = unbounded).  Returns like ``fa_fwd``."""
    pr = _problem(q, k, causal, scale, window)
    B, H, N, d = _shape(q)
    _same(q, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(k, v, dtype=torch.bfloat16, shape=(B, pr.H_kv, N, d))
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if o_resid is None and save_residual:
        o_resid = torch.empty_like(q)
    _same(o, dtype=torch.bfloat16, shape=(B, H, N, d))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    if workspace is None:
        workspace = torch.empty(max(fa_attn_fwd_workspace_size(pr), 1), dtype=torch.uint8, device=q.device)
    st = library().fa_attn_fwd(ctypes.byref(pr), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                               lse.data_ptr(), None if o_resid is None else o_resid.data_ptr(), workspace.data_ptr(),
                               workspace.numel(), _stream_handle(stream))
    _check("fa_attn_fwd", st)
    return (o, lse) if o_resid is None else (o, lse, o_resid)


def fa_attn_fwd_fp8_workspace_size(problem: FaAttnProblem) -> int:
    return int(library().fa_attn_fwd_fp8_workspace_size(ctypes.byref(problem)))


def fa_attn_fwd_fp8(q, k, v, q_descale: float, k_descale: float, v_descale: float, causal: bool = False,
                    scale: float | None = None, window=(-1, -1), o=None, lse=None, workspace=None, stream=None):
    """8-bit forward: q (B, H, N, d), k and v (B, H_kv, N, d) ``torch.float8_e4m3fn`` CUDA
    tensors holding Q / q_descale etc. (per-tensor descales, d = 128 or 64).  Computes the
    attention of the dequantized inputs; returns (o bf16, lse fp32)."""
    pr = _problem(q, k, causal, scale, window)
    B, H, N, d = _shape(q)
    _same(q, dtype=torch.float8_e4m3fn, shape=(B, H, N, d))
    _same(k, v, dtype=torch.float8_e4m3fn, shape=(B, pr.H_kv, N, d))
    if o is None:
        o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _same(o, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    if workspace is None:
        workspace = torch.empty(max(fa_attn_fwd_fp8_workspace_size(pr), 1), dtype=torch.uint8, device=q.device)
    st = library().fa_attn_fwd_fp8(ctypes.byref(pr), q.data_ptr(), k.data_ptr(), v.data_ptr(), float(q_descale),
                                   float(k_descale), float(v_descale), o.data_ptr(), lse.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    _check("fa_attn_fwd_fp8", st)
    return o, lse


def fa_attn_bwd(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None, window=(-1, -1),
                workspace=None, dq=None, dk=None, dv=None, o_resid=None, stream=None):
    """Backward with every option (the same problem as the forward).  Returns (dq, dk, dv)."""
    pr = _problem(q, k, causal, scale, window)
    B, H, N, d = _shape(q)
    _same(q, o, do, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(k, v, dtype=torch.bfloat16, shape=(B, pr.H_kv, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    if dq is None:
        dq = torch.empty((B, H, N, d), dtype=torch.float32, device=q.device)
    if dk is None:
        dk = torch.empty((B, pr.H_kv, N, d), dtype=torch.float32, device=q.device)
    if dv is None:
        dv = torch.empty_like(dk)
    _same(dq, dtype=torch.float32, shape=(B, H, N, d))
    _same(dk, dv, dtype=torch.float32, shape=(B, pr.H_kv, N, d))
    if workspace is None:
        workspace = torch.empty(max(fa_attn_bwd_workspace_size(pr), 1), dtype=torch.uint8, device=q.device)
    st = library().fa_attn_bwd(ctypes.byref(pr), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                               None if o_resid is None else o_resid.data_ptr(), do.data_ptr(), lse.data_ptr(),
                               dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), workspace.numel(),
                               _stream_handle(stream))
    _check("fa_attn_bwd", st)
    return dq, dk, dv


def fa_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, causal: bool = False, scale: float | None = None,
                   o_resid=None, stream=None):
    """The backward pass without a workspace, for callers that cannot allocate device memory
    when they run it: the C entry point uses a scratch array built into the library (64 MiB
    per GPU, shared by all calls on that GPU, so overlapping calls race).  The caller passes
    every input and the fp32 outputs dq, dk, dv; nothing is allocated here either."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, do, dtype=torch.bfloat16, shape=(B, H, N, d))
    _same(lse, dtype=torch.float32, shape=(B, H, N))
    _same(dq, dk, dv, dtype=torch.float32, shape=(B, H, N, d))
    if o_resid is not None:
        _same(o_resid, dtype=torch.bfloat16, shape=(B, H, N, d))
    st = library().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  None if o_resid is None else o_resid.data_ptr(), do.data_ptr(), lse.data_ptr(),
                                  dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, _scale(scale, d),
                                  int(bool(causal)), _stream_handle(stream))
    _check("fa_bwd_noalloc", st)
    return dq, dk, dv


# ---- paged key/value cache.  These calls run on the tensors' device whatever the current one is.
# With ``stream`` left out they run on that device's current stream; what they allocate themselves
# belongs to the stream they run on.

_PAGED_DTYPES = {torch.bfloat16: FA_BF16, torch.float16: FA_F16}
# fa_paged_problem, fa_page_table and fa_page_planes as bytes: a quarter of the time of filling in a
# ctypes structure, in calls that take the GPU a few microseconds
_PROBLEM = struct.Struct("@12if6q")
_TABLE = struct.Struct("@5i3P")
_PLANES = struct.Struct("@P2i2q")
assert (_PROBLEM.size, _TABLE.size, _PLANES.size) == tuple(
    ctypes.sizeof(t) for t in (FaPagedProblem, FaPageTable, FaPagePlanes))
# the handle alone where torch offers it: 0.1 us, a Stream object takes 3 us of a call that runs for 10 us
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch_on(device: torch.device, stream, fn, *args) -> int:
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _launch_on(device, stream, fn, *args)
    if stream is None:
        return fn(*args, _current_stream(device.index))
    if getattr(stream, "device", device) != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return fn(*args, _stream_handle(stream))


def _empty_for(stream, shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """An array for work on ``stream``: it is not handed out again before that work is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        if not stream:  # the legacy default stream
            stream = torch.cuda.default_stream(device)
        else:
            stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _cuda_device(t: torch.Tensor) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("expected CUDA tensors")
    return t.device


def _int32(name: str, t: torch.Tensor, device: torch.device, size: int | None = None) -> int:
    """Address of a dense 1-D int32 array on ``device``."""
    if t.dtype != torch.int32 or t.dim() != 1 or t.device != device or not t.is_contiguous() or \
            (size is not None and t.numel() != size):
        what = "" if size is None else f" of {size} elements"
        raise ValueError(f"{name}: expected a contiguous 1-D int32 tensor{what} on {device}")
    return t.data_ptr()


def _dense(name: str, t: torch.Tensor, dtype: torch.dtype, shape, device: torch.device) -> int:
    """Address of a dense array of that type and shape on ``device``."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _workspace_args(workspace: torch.Tensor, device: torch.device) -> tuple[int, int]:
    if workspace.device != device:
        raise ValueError(f"expected the workspace on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _table_dims(block_table: torch.Tensor, device: torch.device) -> tuple[int, int, int]:
    """rows, max_pages and the row stride of a block table."""
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.device != device:
        raise ValueError(f"block_table: expected a 2-D int32 tensor on {device}")
    rows, width = block_table.shape
    step, one = block_table.stride()
    if rows <= 1:
        step = width
    if (width > 1 and one != 1) or step < width:
        raise ValueError("block_table: the entries of a row must lie side by side and rows must not overlap")
    return rows, width, step


def _pool_strides(pool: torch.Tensor, shape) -> tuple[int, int, int]:
    """Elements between pages, heads and tokens of a (num_pages, H_kv, page_size, d) pool."""
    pages, heads, ps, d = shape
    page, head, token, one = pool.stride()
    if not pages * heads * ps * d:
        return heads * ps * d, ps * d, d
    if d > 1 and one != 1:
        raise ValueError("pages: the d elements of a token must lie side by side")
    if ps == 1:  # the stride of a dimension of one element says nothing
        token = d
    if heads == 1:
        head = ps * token
    if pages == 1:
        page = heads * ps * d
    return page, head, token


def _paged(q: torch.Tensor, k_pages, v_pages, block_table, shape, H: int, H_kv: int, prefix_len, causal, scale,
           device: torch.device) -> bytes:
    """``fa_paged_problem`` of these tensors; ``shape`` is q's."""
    dtype = q.dtype
    if dtype not in _PAGED_DTYPES:
        raise ValueError("expected bf16 or fp16 tensors")
    B, _, T, d = shape
    pool = k_pages.shape
    if len(pool) != 4 or v_pages.shape != pool or pool[1] != H_kv or pool[3] != d:
        raise ValueError("k_pages and v_pages must be (num_pages, H_kv, page_size, d)")
    if k_pages.dtype != dtype or v_pages.dtype != dtype or k_pages.device != device or v_pages.device != device:
        raise ValueError(f"expected pages of {dtype} on {device}")
    rows, width, step = _table_dims(block_table, device)
    if rows != B:
        raise ValueError(f"block_table has {rows} rows for {B} sequences")
    k_stride = _pool_strides(k_pages, pool)
    v_stride = _pool_strides(v_pages, pool)
    try:
        return _PROBLEM.pack(B, H, H_kv, T, d, _PAGED_DTYPES[dtype], pool[2], pool[0], width, step, prefix_len,
                             1 if causal else 0, d ** -0.5 if scale is None else scale, *k_stride, *v_stride)
    except struct.error as e:
        raise ValueError(f"sizes beyond 32 bits, or no numbers: {e}") from None


def _attn_problem(q, k_pages, v_pages, block_table, shape, prefix_len, causal, scale, device) -> bytes:
    if len(shape) != 4:
        raise ValueError("expected a (B, H, T, d) tensor")
    H = shape[1]
    H_kv = k_pages.shape[1] if k_pages.dim() == 4 else 0
    if H_kv < 1 or H % H_kv:
        raise ValueError("k_pages must be (num_pages, H_kv, page_size, d), q's head count a multiple of H_kv")
    return _paged(q, k_pages, v_pages, block_table, shape, H, H_kv, prefix_len, causal, scale, device)


def paged_problem(q, k_pages, v_pages, block_table, prefix_len: int = 0, causal: bool = True,
                  scale: float | None = None) -> FaPagedProblem:
    """The ``fa_paged_problem`` of these tensors (as ``fa_paged_attn`` takes them)."""
    return FaPagedProblem.from_buffer_copy(
        _attn_problem(q, k_pages, v_pages, block_table, q.shape, prefix_len, causal, scale, _cuda_device(q)))


def fa_paged_attn_workspace_size(problem: FaPagedProblem) -> int:
    return int(library().fa_paged_attn_workspace_size(ctypes.byref(problem)))


def fa_paged_attn(q, k_pages, v_pages, block_table, seq_lens, prefix_table=None, prefix_len: int = 0,
                  causal: bool = True, scale: float | None = None, o=None, lse=None, workspace=None, stream=None):
    """Attention of the newest T tokens of every sequence over a paged cache (C ``fa_paged_attn``).

    q (B, H, T, d) bf16 or fp16; k_pages, v_pages (num_pages, H_kv, page_size, d) with any strides
    that keep a token's d elements together; block_table (B, max_pages) and seq_lens (B) int32;
    prefix_table int32 with the pages of ``prefix_len`` tokens that all sequences share.  Returns
    (o, lse).  Rows of negative length are left as they are in ``o`` and ``lse``."""
    device, shape = _cuda_device(q), q.shape
    pr = _attn_problem(q, k_pages, v_pages, block_table, shape, prefix_len, causal, scale, device)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    lens = _int32("seq_lens", seq_lens, device, shape[0])
    prefix = None
    if prefix_len > 0:
        if prefix_table is None:
            raise ValueError("prefix_len needs a prefix_table")
        prefix = _int32("prefix_table", prefix_table, device)
        if prefix_table.numel() * k_pages.shape[2] < prefix_len:
            raise ValueError(f"prefix_table has {prefix_table.numel()} pages for {prefix_len} tokens")
    if o is None:
        o = _empty_for(stream, shape, q.dtype, device)
    if lse is None:
        lse = _empty_for(stream, shape[:3], torch.float32, device)
    if workspace is None:
        workspace = _empty_for(stream, max(library().fa_paged_attn_workspace_size(pr), 1), torch.uint8, device)
    st = _launch_on(device, stream, library().fa_paged_attn, pr, q.data_ptr(), k_pages.data_ptr(),
                    v_pages.data_ptr(), block_table.data_ptr(), lens, prefix, _dense("o", o, q.dtype, shape, device),
                    _dense("lse", lse, torch.float32, shape[:3], device), *_workspace_args(workspace, device))
    if st != FA_OK:
        raise FAError("fa_paged_attn", st)
    return o, lse


def fa_pages_write(k, v, k_pages, v_pages, block_table, seq_lens, stream=None) -> None:
    """Put k, v (B, H_kv, T, d), the T newest tokens of every sequence, into their pages (C
    ``fa_pages_write``): token t of row b goes to position seq_lens[b] - T + t."""
    device, shape = _cuda_device(k), k.shape
    if len(shape) != 4:
        raise ValueError("expected (B, H_kv, T, d) tensors")
    pr = _paged(k, k_pages, v_pages, block_table, shape, shape[1], shape[1], 0, True, 1.0, device)
    st = _launch_on(device, stream, library().fa_pages_write, pr, _dense("k", k, k.dtype, shape, device),
                    _dense("v", v, k.dtype, shape, device), k_pages.data_ptr(), v_pages.data_ptr(),
                    block_table.data_ptr(), _int32("seq_lens", seq_lens, device, shape[0]))
    if st != FA_OK:
        raise FAError("fa_pages_write", st)


def fa_pages_workspace_size(rows: int, num_pages: int) -> int:
    return int(library().fa_pages_workspace_size(rows, num_pages))


def _planes(planes) -> tuple[bytes, object, torch.device]:
    """``fa_page_planes`` (and the array of addresses that it points to) of one (n_planes,
    num_pages, ...) tensor or of a sequence of (num_pages, ...) tensors of one shape, type and
    layout; each page is dense."""
    if isinstance(planes, torch.Tensor):
        x, shape, strides = planes, planes.shape[1:], planes.stride()[1:]
        if planes.dim() < 3 or not planes.shape[0]:
            raise ValueError("planes: expected a (n_planes, num_pages, ...) tensor")
        esize = x.element_size()
        apart, first = planes.stride(0) * esize, planes.data_ptr()
        ptrs = [first + i * apart for i in range(planes.shape[0])]
    else:
        tensors = list(planes)
        if not tensors:
            raise ValueError("planes: expected at least one plane")
        x = tensors[0]
        _cuda_device(x)
        shape, strides, dtype, where = x.shape, x.stride(), x.dtype, x.device
        if len(shape) < 2:
            raise ValueError("planes: expected (num_pages, ...) tensors")
        for t in tensors:
            if t.shape != shape or t.dtype != dtype or t.stride() != strides or t.device != where:
                raise ValueError("planes: expected tensors of one shape, type, layout and device")
        esize = x.element_size()
        ptrs = [t.data_ptr() for t in tensors]
    size = 1
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] > 1 and strides[i] != size:
            raise ValueError("planes: the elements of a page must lie side by side")
        size *= shape[i]
    pages = shape[0]
    step = strides[0] if pages > 1 else size
    if not size:  # strides and addresses of empty tensors say nothing
        step, ptrs = 0, [None] * len(ptrs)
    if step < size:
        raise ValueError("planes: pages must not overlap")
    device = _cuda_device(x)
    array = (ctypes.c_void_p * len(ptrs))(*ptrs)
    return _PLANES.pack(ctypes.addressof(array), len(ptrs), pages, size * esize, step * esize), array, device


def _page_table(page_size: int, block_table, seq_lens, ref_counts) -> tuple[bytes, torch.device]:
    device = _cuda_device(block_table)
    rows, width, step = _table_dims(block_table, device)
    return _TABLE.pack(rows, width, step, page_size, ref_counts.numel(), block_table.data_ptr(),
                       _int32("seq_lens", seq_lens, device, rows),
                       _int32("ref_counts", ref_counts, device)), device


def _pages_workspace(workspace, seq_lens, ref_counts, device: torch.device, stream) -> torch.Tensor:
    if workspace is None:
        return _empty_for(stream, fa_pages_workspace_size(seq_lens.numel(), ref_counts.numel()), torch.uint8, device)
    return workspace


def fa_pages_copy(planes, src, dst, stream=None) -> None:
    """Page dst[i] = page src[i] in every plane (C ``fa_pages_copy``).  planes: one (n_planes,
    num_pages, ...) tensor, or a sequence of (num_pages, ...) tensors (K and V of every layer)."""
    pl, array, device = _planes(planes)  # (the array lives until the call is over)
    n = src.numel()
    st = _launch_on(device, stream, library().fa_pages_copy, pl, _int32("src", src, device),
                    _int32("dst", dst, device, n), n)
    _check("fa_pages_copy", st)


def fa_pages_reserve(page_size: int, block_table, seq_lens, ref_counts, new_lens, workspace=None, stream=None) -> None:
    """Pages for new_lens[b] tokens of every row b (C ``fa_pages_reserve``); updates block_table,
    seq_lens and ref_counts."""
    table, device = _page_table(page_size, block_table, seq_lens, ref_counts)
    lens = _int32("new_lens", new_lens, device, seq_lens.numel())
    ws = _pages_workspace(workspace, seq_lens, ref_counts, device, stream)
    st = _launch_on(device, stream, library().fa_pages_reserve, table, lens,
                    *_workspace_args(ws, device))
    _check("fa_pages_reserve", st)


def fa_pages_fork(planes, page_size: int, block_table, seq_lens, ref_counts, parents, children, workspace=None,
                  stream=None) -> None:
    """Row children[i] continues from row parents[i] (C ``fa_pages_fork``): full pages are shared,
    a partly filled last page is copied in every plane (planes as for ``fa_pages_copy``)."""
    pl, array, device = _planes(planes)
    table, table_device = _page_table(page_size, block_table, seq_lens, ref_counts)
    if table_device != device:
        raise ValueError(f"expected the table on {device}")
    n = parents.numel()
    ws = _pages_workspace(workspace, seq_lens, ref_counts, device, stream)
    st = _launch_on(device, stream, library().fa_pages_fork, pl, table,
                    _int32("parents", parents, device), _int32("children", children, device, n), n,
                    *_workspace_args(ws, device))
    _check("fa_pages_fork", st)


def fa_pages_free(page_size: int, block_table, seq_lens, ref_counts, rows, stream=None) -> None:
    """Take back the pages of the given rows (C ``fa_pages_free``)."""
    table, device = _page_table(page_size, block_table, seq_lens, ref_counts)
    st = _launch_on(device, stream, library().fa_pages_free, table, _int32("rows", rows, device),
                    rows.numel())
    _check("fa_pages_free", st)


def fa_pages_compact(planes, page_size: int, block_table, seq_lens, ref_counts, block_table_out=None,
                     ref_counts_out=None, page_map=None, workspace=None, stream=None):
    """Move the live pages to the front of the pool (C ``fa_pages_compact``; planes as for
    ``fa_pages_copy``).  Returns (block_table_out, ref_counts_out, page_map); the first two may be
    block_table and ref_counts themselves."""
    pl, array, device = _planes(planes)
    table, table_device = _page_table(page_size, block_table, seq_lens, ref_counts)
    if table_device != device:
        raise ValueError(f"expected the table on {device}")
    rows, width, step = _table_dims(block_table, device)
    pages = ref_counts.numel()
    if block_table_out is None:
        block_table_out = _empty_for(stream, (rows, step), torch.int32, device)[:, :width]
    if ref_counts_out is None:
        ref_counts_out = _empty_for(stream, pages, torch.int32, device)
    if page_map is None:
        page_map = _empty_for(stream, pages, torch.int32, device)
    out_rows, out_width, out_step = _table_dims(block_table_out, device)
    if (out_rows, out_width) != (rows, width) or (rows > 1 and out_step != step):
        raise ValueError("block_table_out: expected the shape and row stride of block_table")
    ws = _pages_workspace(workspace, seq_lens, ref_counts, device, stream)
    st = _launch_on(device, stream, library().fa_pages_compact, pl, table,
                    block_table_out.data_ptr(), _int32("ref_counts_out", ref_counts_out, device, pages),
                    _int32("page_map", page_map, device, pages), *_workspace_args(ws, device))
    _check("fa_pages_compact", st)
    return block_table_out, ref_counts_out, page_map


def fa_selftest_wait_timeout(stream=None) -> None:
    """Enqueue the bounded-wait self-test (a wait that must give up after ~2 s and report
    FA_ERR_TIMEOUT through ``fa_device_status``)."""
    _check("fa_selftest_wait_timeout", library().fa_selftest_wait_timeout(_stream_handle(stream)))


def fa_selftest_paged_give_up(q, k_pages, v_pages, block_table, seq_lens, prefix_table, prefix_len: int, o, lse,
                              workspace, segment: int, causal: bool = True, stream=None) -> None:
    """Enqueue ``fa_paged_attn`` with waits that give up from a CTA's part ``segment`` (>= 1) on (C
    ``fa_selftest_paged_give_up``)."""
    device, shape = _cuda_device(q), q.shape
    pr = _attn_problem(q, k_pages, v_pages, block_table, shape, prefix_len, causal, None, device)
    ws, ws_bytes = _workspace_args(workspace, device)
    _check("fa_selftest_paged_give_up", _launch_on(
        device, stream, library().fa_selftest_paged_give_up, pr, _dense("q", q, q.dtype, shape, device),
        k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), _int32("seq_lens", seq_lens, device, shape[0]),
        None if prefix_table is None else _int32("prefix_table", prefix_table, device),
        _dense("o", o, q.dtype, shape, device), _dense("lse", lse, torch.float32, shape[:3], device), ws, ws_bytes,
        segment))


def fa_selftest_exp2(x: torch.Tensor, stream=None) -> torch.Tensor:
    """The FMA-pipe exponential of the softmax kernels applied to a 1-D fp32 CUDA tensor."""
    if x.dtype != torch.float32 or x.dim() != 1 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError("expected a contiguous 1-D fp32 CUDA tensor")
    y = torch.empty_like(x)
    _check("fa_selftest_exp2", library().fa_selftest_exp2(x.data_ptr(), y.data_ptr(), x.numel(),
                                                          _stream_handle(stream)))
    return y


def fa_last_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the device status code: FA_OK, FA_ERR_TIMEOUT,
    FA_ERR_RANGE, FA_ERR_INDEX, FA_ERR_NO_PAGES or FA_ERR_CUDA."""
    return int(library().fa_last_device_status(_stream_handle(stream)))


def fa_device_status(stream=None) -> int:
    """``fa_last_device_status`` under its earlier name."""
    return int(library().fa_device_status(_stream_handle(stream)))


_PHASE_EVENTS = None  # keeps the ctypes array alive while the hook is set


def fa_bwd_set_phase_events(events=None) -> None:
    """Profiling hook: record ``events[0]`` after the preprocess and ``events[1]`` after the
    dK/dV kernel in every later ``fa_bwd`` of this thread (``torch.cuda.Event`` objects);
    ``None`` turns it off."""
    global _PHASE_EVENTS
    if events is None:
        _PHASE_EVENTS = None
        library().fa_bwd_set_phase_events(None)
        return
    for ev in events[:2]:
        if not ev.cuda_event:  # torch creates the CUDA event lazily, on its first record
            ev.record()
    arr = (ctypes.c_void_p * 2)(events[0].cuda_event, events[1].cuda_event)
    _PHASE_EVENTS = arr
    library().fa_bwd_set_phase_events(ctypes.cast(arr, ctypes.c_void_p))
