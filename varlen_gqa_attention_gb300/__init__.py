"""Length-aware GQA attention over a per-sequence KV column store, for GB300 (sm_103a).

A thin ctypes binding over ``libsdpa_varlen.so`` (C interface in include/sdpa_varlen.h):
it only checks tensor dtypes/devices, reads strides and pointers, allocates outputs and
workspace with torch, and passes the given (else the current) CUDA stream.  Every step of the computation
runs in the library's CUDA kernels; there is no other implementation to fall back on, so a
missing library is an error.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import NamedTuple, Optional, Sequence

import torch

from . import _build

__all__ = [
    "sdpa_varlen", "sdpa_varlen_modes", "sdpa_varlen_append", "sdpa_seq_clone", "sdpa_causal_prefill",
    "sdpa_varlen_splitk_static", "sdpa_rope", "sdpa_rope_append", "sdpa_rope_append_q4", "sdpa_q4_unpack",
    "sdpa_varlen_q4", "Q4Store", "q4_store", "rope_table", "q4_workspace_bytes", "sdpa_rope_append_q8", "sdpa_q8_unpack",
    "sdpa_varlen_q8", "Q8Store", "q8_store", "q8_workspace_bytes", "workspace_bytes", "workspace_status", "prefill_available", "set_route_policy",
    "set_timing_events", "library",
    "SDPA_OK", "SEG_BAD_QRANGE", "SEG_BAD_COL", "SEG_BAD_KV", "SEG_SPAN", "SEG_OVERLAP",
    "DEV_TIMEOUT", "ROPE_BAD_POS", "ROUTE_AUTO", "ROUTE_SPLITK", "ROUTE_PREFILL", "SdpaError",
]

SDPA_OK = 0
SEG_BAD_QRANGE, SEG_BAD_COL, SEG_BAD_KV, SEG_SPAN, SEG_OVERLAP, DEV_TIMEOUT = 1, 2, 4, 8, 16, 32
ROPE_BAD_POS = 64
ROUTE_AUTO, ROUTE_SPLITK, ROUTE_PREFILL = 0, 1, 2

STATUS_NAMES = {
    0: "SDPA_OK", 1: "SDPA_ERR_NULL", 2: "SDPA_ERR_SHAPE", 3: "SDPA_ERR_HEAD_DIM", 4: "SDPA_ERR_GQA",
    5: "SDPA_ERR_STRIDE", 6: "SDPA_ERR_ALIGN", 7: "SDPA_ERR_WORKSPACE", 8: "SDPA_ERR_ARG",
    9: "SDPA_ERR_CUDA",
}

EXPORTS = [
    "sdpa_varlen_workspace_bytes", "sdpa_varlen", "sdpa_causal_prefill", "sdpa_set_route_policy",
    "sdpa_set_timing_events", "sdpa_last_error", "sdpa_version", "sdpa_varlen_splitk_static",
    "sdpa_varlen_append", "sdpa_seq_clone", "sdpa_varlen_modes", "sdpa_prefill_available",
    "sdpa_workspace_status", "sdpa_rope", "sdpa_rope_append", "sdpa_rope_append_fourbit", "sdpa_fourbit_unpack",
    "sdpa_varlen_fourbit", "sdpa_varlen_fourbit_workspace_bytes", "sdpa_rope_append_eightbit", "sdpa_eightbit_unpack",
    "sdpa_varlen_eightbit", "sdpa_varlen_eightbit_workspace_bytes",
]


class SdpaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


# the C structs sdpa_rotation, sdpa_q4_store and sdpa_q8_store, packed (their padding included) as bytes
_ROTATION = struct.Struct("@PqPq7i4x")
_Q4_POINTERS = _Q8_POINTERS = struct.Struct("@4P")


_bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

_lib: Optional[ctypes.CDLL] = None


def library(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libsdpa_varlen.so (building it first when it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.lib_path()
    if not os.path.exists(path):
        if not build_if_missing:
            raise ImportError(f"{path} is missing; run __graft_entry__.build()")
        _build.build()
    lib = ctypes.CDLL(path)
    c_i64, c_int, c_vp, c_f = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
    lib.sdpa_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.sdpa_varlen_workspace_bytes.argtypes = [c_i64, c_int, c_int, c_int, c_int]
    lib.sdpa_varlen.restype = c_int
    lib.sdpa_varlen.argtypes = [c_vp, c_i64, c_int, c_int, c_i64, c_i64, c_vp, c_vp, c_i64, c_int,
                                c_int, c_vp, c_int, c_int, c_int, c_f, c_vp, c_i64, c_i64, c_vp,
                                ctypes.c_size_t, c_vp, c_vp]
    lib.sdpa_varlen_append.restype = c_int
    lib.sdpa_varlen_append.argtypes = [c_vp, c_i64, c_int, c_int, c_i64, c_i64, c_vp, c_vp, c_i64, c_i64,
                                       c_vp, c_vp, c_i64, c_int, c_int, c_vp, c_int, c_int, c_int, c_f,
                                       c_vp, c_i64, c_i64, c_vp, ctypes.c_size_t, c_vp, c_vp]
    lib.sdpa_varlen_modes.restype = c_int
    lib.sdpa_varlen_modes.argtypes = [c_vp, c_i64, c_int, c_int, c_i64, c_i64, c_vp, c_vp, c_i64, c_int,
                                      c_int, c_vp, c_vp, c_int, c_f, c_vp, c_i64, c_i64, c_vp,
                                      ctypes.c_size_t, c_vp, c_vp]
    lib.sdpa_seq_clone.restype = c_int
    lib.sdpa_seq_clone.argtypes = [c_vp, c_vp, c_i64, c_int, c_int, c_int, c_int, c_int, c_i64, c_vp]
    lib.sdpa_causal_prefill.restype = c_int
    lib.sdpa_causal_prefill.argtypes = [c_vp, c_vp, c_vp, c_i64, c_i64, c_int, c_int, c_int, c_f,
                                        c_vp, c_vp, ctypes.c_size_t, c_vp]
    lib.sdpa_set_route_policy.restype = c_int
    lib.sdpa_set_route_policy.argtypes = [c_int]
    lib.sdpa_set_timing_events.restype = c_int
    lib.sdpa_set_timing_events.argtypes = [ctypes.POINTER(c_vp), c_int]
    lib.sdpa_last_error.restype = ctypes.c_char_p
    lib.sdpa_last_error.argtypes = []
    lib.sdpa_prefill_available.restype = c_int
    lib.sdpa_prefill_available.argtypes = [c_int]
    lib.sdpa_version.restype = c_int
    lib.sdpa_version.argtypes = []
    lib.sdpa_varlen_splitk_static.restype = c_int
    lib.sdpa_varlen_splitk_static.argtypes = [c_vp, c_i64, c_int, c_int, c_i64, c_i64, c_vp, c_vp, c_i64, c_int,
                                              c_int, c_vp, c_int, c_int, c_int, c_f, c_vp, c_i64, c_i64, c_vp,
                                              c_vp]
    lib.sdpa_workspace_status.restype = c_int
    lib.sdpa_workspace_status.argtypes = [c_vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32), c_vp]
    c_rot = c_q4 = c_vp  # packed structs (_ROTATION, _Q4_POINTERS)
    lib.sdpa_rope.restype = c_int
    lib.sdpa_rope.argtypes = [c_vp, c_i64, c_int, c_int, c_i64, c_i64, c_rot, c_int, c_vp, c_i64, c_i64, c_vp, c_vp]
    step = [c_vp, c_i64, c_i64] * 3 + [c_i64, c_int, c_int, c_int, c_rot]  # q, k_new, v_new, sizes, rotation
    table = [c_i64, c_int, c_vp, c_vp, c_int, c_int]                       # rows, cols, seq_info .. window
    lib.sdpa_rope_append.restype = c_int
    lib.sdpa_rope_append.argtypes = step + [c_vp, c_vp] + table + [c_vp, c_i64, c_i64, c_vp, c_vp]
    lib.sdpa_rope_append_fourbit.restype = c_int
    lib.sdpa_rope_append_fourbit.argtypes = step + [c_q4] + table + [c_vp, c_i64, c_i64, c_vp, c_vp]
    lib.sdpa_fourbit_unpack.restype = c_int
    lib.sdpa_fourbit_unpack.argtypes = [c_q4, c_i64, c_int, c_int, c_int, c_vp, c_vp, c_int, c_int, c_i64, c_vp, c_vp,
                                   c_i64, c_i64, c_vp, c_vp]
    lib.sdpa_rope_append_eightbit.restype = c_int
    lib.sdpa_rope_append_eightbit.argtypes = lib.sdpa_rope_append_fourbit.argtypes
    lib.sdpa_eightbit_unpack.restype = c_int
    lib.sdpa_eightbit_unpack.argtypes = lib.sdpa_fourbit_unpack.argtypes
    lib.sdpa_varlen_fourbit_workspace_bytes.restype = ctypes.c_size_t
    lib.sdpa_varlen_fourbit_workspace_bytes.argtypes = [c_i64, c_int, c_int, c_int, c_int, c_i64, c_int]
    lib.sdpa_varlen_fourbit.restype = c_int
    lib.sdpa_varlen_fourbit.argtypes = [c_vp, c_i64, c_int, c_int, c_i64, c_i64, c_q4, c_i64, c_int, c_int, c_vp, c_vp,
                                   c_int, c_int, c_int, c_f, c_vp, c_i64, c_i64, c_vp, ctypes.c_size_t, c_vp, c_vp]
    lib.sdpa_varlen_eightbit_workspace_bytes.restype = ctypes.c_size_t
    lib.sdpa_varlen_eightbit_workspace_bytes.argtypes = lib.sdpa_varlen_fourbit_workspace_bytes.argtypes
    lib.sdpa_varlen_eightbit.restype = c_int
    lib.sdpa_varlen_eightbit.argtypes = lib.sdpa_varlen_fourbit.argtypes
    _lib = lib
    return lib


def _check(code: int):
    if code != SDPA_OK:
        raise SdpaError(code, library().sdpa_last_error().decode())


def workspace_bytes(T: int, Hq: int, Hkv: int, D: int, S: int) -> int:
    return int(library().sdpa_varlen_workspace_bytes(T, Hq, Hkv, D, S))


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Status word of the last call that used ``workspace``: its SDPA_SEG_* bits and
    DEV_TIMEOUT.  Waits for the stream, so it is not for use inside graph capture."""
    v = ctypes.c_int32(0)
    _check(library().sdpa_workspace_status(workspace.data_ptr(), workspace.numel(), ctypes.byref(v),
                                           _stream_ptr(stream)))
    return int(v.value)


def prefill_available(D: int) -> bool:
    """Whether the tensor-memory prefill kernel runs for head dim D on the current device."""
    lib = library()
    r = lib.sdpa_prefill_available(D)
    if r < 0:
        raise SdpaError(9 if D in (64, 128, 256) else 3, lib.sdpa_last_error().decode())
    return r == 1


def set_route_policy(policy: int) -> None:
    _check(library().sdpa_set_route_policy(policy))


def set_timing_events(events) -> None:
    """Record 5 torch.cuda.Event objects at the kernel boundaries of this thread's next calls
    (scheduler | prefill | split-K | combine); ``None`` switches the hook off."""
    lib = library()
    if events is None:
        _check(lib.sdpa_set_timing_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib.sdpa_set_timing_events(arr, len(events)))


def _rows_like(like: torch.Tensor, shape, stream) -> torch.Tensor:
    """Uninitialised bf16 rows on `like`'s device, of memory that belongs to the stream that will
    write them.  The current stream's work on them counts too before that memory serves again: the
    caller reads them there."""
    if stream is None:
        return torch.empty(shape, dtype=_bf16, device=like.device)
    with torch.cuda.stream(stream):
        rows = torch.empty(shape, dtype=_bf16, device=like.device)
    rows.record_stream(torch.cuda.current_stream(like.device))
    return rows


def _workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """Workspace for one call, of memory that belongs to the stream that uses it."""
    if stream is None:
        return torch.empty(max(nbytes, 256), dtype=_u8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 256), dtype=_u8, device=device)


def _stream_ptr(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _window(window) -> int:
    """A window as the C entries' 32-bit int, which ctypes would cut larger numbers to."""
    w = int(window)
    if not -2 ** 31 <= w < 2 ** 31:
        raise ValueError(f"window {w} is beyond 32 bits")
    return w


def _check_scratch(q, workspace, status) -> None:
    """What the kernels write beside their output: a caller's workspace and status word."""
    if workspace is not None and (workspace.device != q.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on q's CUDA device")
    if status is not None and (status.dtype != torch.int32 or status.device != q.device or status.numel() < 1):
        raise ValueError("status must be an int32 tensor on q's CUDA device")


def _check_attention_args(q, k_store, v_store, seq_info, out=None, seg_mode=None, workspace=None, status=None):
    """The tensor checks every attention entry makes before its C call: shapes, dtypes
    (bf16 data, int32 tables), layouts (contiguous stores and tables, unit inner strides) and
    one CUDA device for all of them.  Raises ValueError; returns (T, Hq, D, rows, cols, Hkv, S)."""
    if q.dim() != 3 or k_store.dim() != 4 or tuple(v_store.shape) != tuple(k_store.shape):
        raise ValueError("q must be [T, Hq, D] and the stores [rows, cols, Hkv, D]")
    for name, t in (("q", q), ("k_store", k_store), ("v_store", v_store)):
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bf16, not {t.dtype}")
    T, Hq, D = q.shape
    rows, cols, Hkv, Dk = k_store.shape
    if Dk != D:
        raise ValueError("head dims of q and the stores differ")
    if q.stride(2) != 1:
        raise ValueError("q must have unit inner stride")
    if not (k_store.is_contiguous() and v_store.is_contiguous()):
        raise ValueError("k_store and v_store must be contiguous")
    if seq_info.dtype != torch.int32 or not seq_info.is_contiguous() or \
            (seq_info.numel() and (seq_info.dim() != 2 or seq_info.shape[1] != 4)):
        raise ValueError("seq_info must be a contiguous int32 [S, 4] tensor")
    S = seq_info.shape[0] if seq_info.numel() else 0
    if out is not None and (out.dtype != torch.bfloat16 or tuple(out.shape) != (T, Hq, D) or out.stride(2) != 1):
        raise ValueError("out must be bf16 [T, Hq, D] with unit inner stride")
    if seg_mode is not None:
        if seg_mode.dtype != torch.int32 or not seg_mode.is_contiguous() or (S and tuple(seg_mode.shape) != (S, 2)):
            raise ValueError("seg_mode must be a contiguous int32 [S, 2] tensor")
    tensors = [q, k_store, v_store, seq_info] + [t for t in (out, seg_mode) if t is not None]
    if not all(t.is_cuda for t in tensors) or len({t.device for t in tensors}) != 1:
        raise ValueError("every tensor must be on the same CUDA device")
    _check_scratch(q, workspace, status)
    return T, Hq, D, rows, cols, Hkv, S


def sdpa_varlen(q: torch.Tensor, k_store: torch.Tensor, v_store: torch.Tensor, seq_info: torch.Tensor,
                *, causal: bool, window: int = 0, scale: Optional[float] = None,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[T, Hq, D] = length-aware GQA attention of q over the column stores.

    q: bf16 [T, Hq, D] (inner stride 1); k_store, v_store: bf16 [rows, cols, Hkv, D]
    contiguous; seq_info: int32 [S, 4] contiguous on the same device.  ``status`` (an int32
    device tensor, optional) receives the OR of the device status bits.
    """
    T, Hq, D, rows, cols, Hkv, S = _check_attention_args(q, k_store, v_store, seq_info, out, None, workspace,
                                                            status)
    lib = library()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _rows_like(q, (T, Hq, D), stream)
    need = workspace_bytes(T, Hq, Hkv, D, S)
    if workspace is None:
        workspace = _workspace(need, q.device, stream)
    st_ptr = status.data_ptr() if status is not None else None
    code = lib.sdpa_varlen(q.data_ptr(), T, Hq, D, q.stride(0), q.stride(1), k_store.data_ptr(),
                           v_store.data_ptr(), rows, cols, Hkv, seq_info.data_ptr() if S else None,
                           S, int(bool(causal)), _window(window), float(scale), out.data_ptr(),
                           out.stride(0), out.stride(1), workspace.data_ptr(), workspace.numel(),
                           st_ptr, _stream_ptr(stream))
    _check(code)
    return out


def sdpa_varlen_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_store: torch.Tensor,
                       v_store: torch.Tensor, seq_info: torch.Tensor, *, causal: bool, window: int = 0,
                       scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Write the step's keys and values into the stores, then attend (one enqueued call).

    k_new, v_new: bf16 [T, Hkv, D] (inner stride 1), row t the new key / value of packed
    query row t; they go to store row (kv_end - q_len + i) % rows of each live segment's
    column.  The stores are modified in place; everything else is as ``sdpa_varlen``.
    """
    T, Hq, D, rows, cols, Hkv, S = _check_attention_args(q, k_store, v_store, seq_info, out, None, workspace,
                                                            status)
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.device != q.device:
            raise ValueError(f"{name} must be a bf16 tensor on q's CUDA device")
    if tuple(k_new.shape) != (T, Hkv, D) or tuple(v_new.shape) != (T, Hkv, D):
        raise ValueError("k_new and v_new must be [T, Hkv, D]")
    if k_new.stride() != v_new.stride() or k_new.stride(2) != 1:
        raise ValueError("k_new and v_new must share strides, with unit inner stride")
    lib = library()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _rows_like(q, (T, Hq, D), stream)
    if workspace is None:
        workspace = _workspace(workspace_bytes(T, Hq, Hkv, D, S), q.device, stream)
    st_ptr = status.data_ptr() if status is not None else None
    code = lib.sdpa_varlen_append(q.data_ptr(), T, Hq, D, q.stride(0), q.stride(1), k_new.data_ptr(),
                                  v_new.data_ptr(), k_new.stride(0), k_new.stride(1), k_store.data_ptr(),
                                  v_store.data_ptr(), rows, cols, Hkv, seq_info.data_ptr() if S else None,
                                  S, int(bool(causal)), _window(window), float(scale), out.data_ptr(),
                                  out.stride(0), out.stride(1), workspace.data_ptr(), workspace.numel(),
                                  st_ptr, _stream_ptr(stream))
    _check(code)
    return out


def sdpa_varlen_modes(q: torch.Tensor, k_store: torch.Tensor, v_store: torch.Tensor, seq_info: torch.Tensor,
                      seg_mode: torch.Tensor, *, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """``sdpa_varlen`` with a mask mode per segment: seg_mode int32 [S, 2] = (causal, window)
    on the device, in place of the call's causal / window."""
    T, Hq, D, rows, cols, Hkv, S = _check_attention_args(q, k_store, v_store, seq_info, out, seg_mode, workspace,
                                                            status)
    lib = library()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _rows_like(q, (T, Hq, D), stream)
    if workspace is None:
        workspace = _workspace(workspace_bytes(T, Hq, Hkv, D, S), q.device, stream)
    st_ptr = status.data_ptr() if status is not None else None
    code = lib.sdpa_varlen_modes(q.data_ptr(), T, Hq, D, q.stride(0), q.stride(1), k_store.data_ptr(),
                                 v_store.data_ptr(), rows, cols, Hkv, seq_info.data_ptr() if S else None,
                                 seg_mode.data_ptr() if S else None, S, float(scale), out.data_ptr(),
                                 out.stride(0), out.stride(1), workspace.data_ptr(), workspace.numel(),
                                 st_ptr, _stream_ptr(stream))
    _check(code)
    return out


def sdpa_seq_clone(k_store: torch.Tensor, v_store: torch.Tensor, src_col: int, dst_col: int, n: int,
                   stream=None) -> None:
    """Column dst_col of both stores takes over the first n positions of column src_col
    (ring-aware: store rows [0, min(n, rows)) are copied).  In place, on the device."""
    lib = library()
    if k_store.dim() != 4 or tuple(v_store.shape) != tuple(k_store.shape):
        raise ValueError("the stores must both be [rows, cols, Hkv, D]")
    for name, t in (("k_store", k_store), ("v_store", v_store)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    if k_store.device != v_store.device:
        raise ValueError("the stores must be on the same CUDA device")
    rows, cols, Hkv, D = k_store.shape
    _check(lib.sdpa_seq_clone(k_store.data_ptr(), v_store.data_ptr(), rows, cols, Hkv, D, int(src_col),
                              int(dst_col), int(n), _stream_ptr(stream)))


def sdpa_causal_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
                        *, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Dense causal GQA attention: q [Lq, Hq, D] against k, v [Lkv, Hkv, D], queries being
    the last Lq positions.  All tensors contiguous bf16 on one CUDA device."""
    lib = library()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous 3-d bf16 CUDA tensor")
    Lq, Hq, D = q.shape
    Lkv, Hkv, Dk = k.shape
    if v.shape != k.shape or Dk != D:
        raise ValueError("k and v must both be [Lkv, Hkv, D], with q's D")
    if k.device != q.device or v.device != q.device:
        raise ValueError("every tensor must be on the same CUDA device")
    if out is not None and (out.dtype != torch.bfloat16 or out.shape != q.shape or out.device != q.device or
                            not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 tensor of q's shape on its CUDA device")
    _check_scratch(q, workspace, None)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _rows_like(q, q.shape, stream)
    need = workspace_bytes(Lq, Hq, Hkv, D, 1)
    if workspace is None:
        workspace = _workspace(need, q.device, stream)
    code = lib.sdpa_causal_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), Lq, Lkv, Hq, Hkv, D,
                                   float(scale), out.data_ptr(), workspace.data_ptr(),
                                   workspace.numel(), _stream_ptr(stream))
    _check(code)
    return out


def sdpa_varlen_splitk_static(q: torch.Tensor, k_store: torch.Tensor, v_store: torch.Tensor,
                              seq_info: torch.Tensor, *, causal: bool, window: int = 0,
                              scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                              status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """sdpa_varlen for callers that cannot allocate device scratch: the library's own static
    device array (SDPA_STATIC_SCRATCH_BYTES) serves as the workspace and every segment runs on
    the split-K kernel.  Pass ``out`` to allocate nothing at all.  Calls must not overlap on
    the GPU (they share the array); make the first call on a device outside stream capture.
    The tensors are checked as for ``sdpa_varlen``."""
    T, Hq, D, rows, cols, Hkv, S = _check_attention_args(q, k_store, v_store, seq_info, out, None, None, status)
    lib = library()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _rows_like(q, (T, Hq, D), stream)
    code = lib.sdpa_varlen_splitk_static(
        q.data_ptr(), T, Hq, D, q.stride(0), q.stride(1), k_store.data_ptr(), v_store.data_ptr(), rows, cols, Hkv,
        seq_info.data_ptr() if S else None, S, int(bool(causal)), _window(window), float(scale), out.data_ptr(),
        out.stride(0), out.stride(1), status.data_ptr() if status is not None else None, _stream_ptr(stream))
    _check(code)
    return out


# ------------------------------------------------ rotary positions and the 4-bit column store
#
# A decode step calls these once a layer and its kernels take a few microseconds, so the checks read
# each tensor's attributes once and the device and stream come as plain numbers.

def _device_of(*tensors) -> int:
    """Index of the one CUDA device that every tensor given is on (None passes)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("every tensor must be on the same CUDA device")
    if dev < 0:
        raise ValueError("every tensor must be on a CUDA device")
    return dev


def _call(entry, dev: int, stream, *args) -> None:
    """Calls a C entry with device `dev` current and its stream (the given one, else the device's
    current one) as the last argument."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"the stream is on device {stream.device_index}, the tensors on {dev}")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        code = entry(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = entry(*args, handle)
    if code != SDPA_OK:
        _check(code)


def _strides(name: str, t: torch.Tensor, shape=None):
    """Row and head strides of bf16 rows [T, heads, D], checked against `shape` when it is given."""
    strides = t.stride()
    if t.dtype is not _bf16 or len(strides) != 3:
        raise ValueError(f"{name} must be bf16 [T, heads, D], not {t.dtype} {list(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if strides[2] != 1:
        raise ValueError(f"{name} must have unit inner stride")
    return strides[0], strides[1]


def _status_ptr(status: Optional[torch.Tensor]):
    if status is None:
        return None
    if status.dtype is not _i32 or status.numel() < 1:
        raise ValueError("status must be an int32 tensor")
    return status.data_ptr()


def _table(seq_info: torch.Tensor, seg_mode: Optional[torch.Tensor]):
    """(seq_info pointer, seg_mode pointer, segments) of a segment table."""
    shape = seq_info.shape
    S = shape[0] if shape else 0
    if seq_info.dtype is not _i32 or not seq_info.is_contiguous() or \
            (len(shape) != 2 or shape[1] != 4) and seq_info.numel():
        raise ValueError("seq_info must be a contiguous int32 [S, 4] tensor")
    if seg_mode is not None:
        if seg_mode.dtype is not _i32 or not seg_mode.is_contiguous() or (S and seg_mode.shape != (S, 2)):
            raise ValueError("seg_mode must be a contiguous int32 [S, 2] tensor")
    if not S or len(shape) != 2 or shape[1] != 4:
        return None, None, 0
    return seq_info.data_ptr(), None if seg_mode is None else seg_mode.data_ptr(), S


def _rotation(table: torch.Tensor, positions: Optional[torch.Tensor], sections: Optional[Sequence[int]],
              interleaved: bool, T: int) -> bytes:
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2 or table.dtype is not _f32 or not table.is_contiguous():
        raise ValueError("table must be contiguous fp32 [positions, rotated pairs, 2]")
    P, half, _ = shape
    if sections is None:
        sections, axes = (half,), 1
    else:
        axes = len(sections)
        if not 1 <= axes <= 4:
            raise ValueError(f"sections has {axes} position axes: 1 to 4")
    ptr = stride = 0
    if positions is not None:
        shape = positions.shape
        if positions.dtype is not _i32 or not (shape == (axes, T) or (axes == 1 and shape == (T,))) or \
                (T > 1 and positions.stride(-1) != 1):
            raise ValueError(f"positions must be int32 [{axes}, {T}] with unit inner stride")
        ptr, stride = positions.data_ptr(), positions.stride(0) if axes > 1 else 0
    elif axes > 1:
        raise ValueError("several position axes need positions")
    return _ROTATION.pack(table.data_ptr(), P, ptr, stride, 2 * half, axes, *sections, *(0,) * (4 - axes),
                          1 if interleaved else 0)


def rope_table(positions: int, rot_dims: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """A rotation table fp32 [positions, rot_dims / 2, 2]: cos and sin of p * base ** (-2 j / rot_dims),
    taken in 64 bits (a far position's angle needs them).  rot_dims: a multiple of 16, as the entries
    take it.  A program makes it once."""
    if rot_dims <= 0 or rot_dims % 16:
        raise ValueError(f"rot_dims must be a positive multiple of 16, not {rot_dims}")
    j = torch.arange(rot_dims // 2, dtype=torch.float64, device=device)
    p = torch.arange(positions, dtype=torch.float64, device=device)
    a = p[:, None] * base ** (-2.0 * j / rot_dims)
    return torch.stack([a.cos(), a.sin()], dim=-1).float()


def sdpa_rope(x: torch.Tensor, table: torch.Tensor, positions: torch.Tensor, *,
              sections: Optional[Sequence[int]] = None, interleaved: bool = False, inverse: bool = False,
              out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """out[T, H, D] = the rows x turned by the angles of their positions.

    x: bf16 [T, H, D] (inner stride 1; ``out`` may be x).  table: fp32 [P, pairs, 2] (cos, sin), the
    first 2 * pairs dims are turned.  positions: int32 [T], or [axes, T] with ``sections`` = the
    number of pairs of each axis (for example time, height and width).  Pairs are dims
    (j, j + pairs), or (2j, 2j + 1) when ``interleaved``.  ``inverse`` turns the other way: the
    gradient.  No autograd graph is kept: a training step turns the output's gradient back with the
    same positions and ``inverse``, in a ``torch.autograd.Function`` of its own or by hand, and an x
    that requires a gradient is refused while gradients are recorded.  Rows with a position outside the table are 0 and set ROPE_BAD_POS in ``status``."""
    rs, hs = _strides("x", x)
    shape = x.shape
    T, H, D = shape
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError("x requires a gradient, and no graph is kept: rotate x.detach(), and its gradient by inverse")
    if positions is None:
        raise ValueError("positions must be given")
    rot = _rotation(table, positions, sections, interleaved, T)
    ors, ohs = _strides("out", out, shape) if out is not None else (H * D, D)
    dev = _device_of(x, table, positions, out, status)
    if out is None:
        out = _rows_like(x, shape, stream)
    _call(library().sdpa_rope, dev, stream, x.data_ptr(), T, H, D, rs, hs, rot, 1 if inverse else 0, out.data_ptr(),
          ors, ohs, _status_ptr(status))
    return out


class Q4Store(NamedTuple):
    """A 4-bit column store: uint8 codes [cols, Hkv, rows, D / 2] and scales [cols, Hkv, rows, D / 32]
    of the keys, then of the values.  Nibble c (byte i: dim 2i low, dim 2i + 1 high) under scale byte b
    stands for (c - 8) * 2**((b >> 3) - 21) * (1 + (b & 7) / 8)."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def q4_store(rows: int, cols: int, Hkv: int, D: int, device=None) -> Q4Store:
    """An empty 4-bit store (every value 0); rows a multiple of 16."""
    if rows <= 0 or rows % 16 or cols <= 0 or Hkv <= 0 or D not in (64, 128, 256):
        raise ValueError("rows must be a multiple of 16, D 64, 128 or 256")
    codes = lambda: torch.full((cols, Hkv, rows, D // 2), 0x88, dtype=_u8, device=device)  # noqa: E731
    scales = lambda: torch.zeros((cols, Hkv, rows, D // 32), dtype=_u8, device=device)  # noqa: E731
    return Q4Store(codes(), scales(), codes(), scales())


def _q4(store: Q4Store):
    """(rows, cols, Hkv, D, packed pointers) of a 4-bit store."""
    kc, ks, vc, vs = store
    shape = kc.shape
    if len(shape) != 4 or vc.shape != shape or ks.shape != vs.shape or \
            ks.shape != (shape[0], shape[1], shape[2], shape[3] // 16):
        raise ValueError("a 4-bit store is codes [cols, Hkv, rows, D / 2] and scales [cols, Hkv, rows, D / 32], twice")
    if not (kc.dtype is ks.dtype is vc.dtype is vs.dtype is _u8 and kc.is_contiguous() and ks.is_contiguous() and
            vc.is_contiguous() and vs.is_contiguous()):
        raise ValueError("a 4-bit store's tensors must be contiguous uint8")
    cols, Hkv, rows, half = shape
    return rows, cols, Hkv, 2 * half, _Q4_POINTERS.pack(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr())


def _rope_append(entry, q, k_new, v_new, store_tensors, store_args, rows, cols, Hkv, D, seq_info, table, positions,
                 sections, interleaved, window, seg_mode, q_out, status, stream):
    qrs, qhs = _strides("q", q)
    shape = q.shape
    T, Hq, Dq = shape
    if Dq != D:
        raise ValueError("head dims of q and the store differ")
    krs, khs = _strides("k_new", k_new, (T, Hkv, D))
    vrs, vhs = _strides("v_new", v_new, (T, Hkv, D))
    seq_ptr, mode_ptr, S = _table(seq_info, seg_mode)
    rot = _rotation(table, positions, sections, interleaved, T)
    ors, ohs = _strides("q_out", q_out, shape) if q_out is not None else (Hq * D, D)
    dev = _device_of(q, k_new, v_new, *store_tensors, seq_info, table, positions, seg_mode, q_out, status)
    if q_out is None:
        q_out = _rows_like(q, shape, stream)
    _call(entry, dev, stream, q.data_ptr(), qrs, qhs, k_new.data_ptr(), krs, khs, v_new.data_ptr(), vrs, vhs, T, Hq,
          Hkv, D, rot, *store_args, rows, cols, seq_ptr, mode_ptr, S, _window(window), q_out.data_ptr(), ors, ohs,
          _status_ptr(status))
    return q_out


def sdpa_rope_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_store: torch.Tensor,
                     v_store: torch.Tensor, seq_info: torch.Tensor, table: torch.Tensor, *,
                     positions: Optional[torch.Tensor] = None, sections: Optional[Sequence[int]] = None,
                     interleaved: bool = False, window: int = 0, seg_mode: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """A step's rows on their way to ``sdpa_varlen``: returns the rotated queries; rotated keys and
    the values go into the bf16 column stores (in place).

    q: bf16 [T, Hq, D]; k_new, v_new: bf16 [T, Hkv, D], each with its own strides.  The rotation is
    ``sdpa_rope``'s; with ``positions`` None a row's position is its place in its sequence.
    ``window`` / ``seg_mode``: as for the attention that follows (they decide which segments are
    valid).  Rows of no live segment: q_out 0, nothing stored."""
    shape = k_store.shape
    if len(shape) != 4 or v_store.shape != shape:
        raise ValueError("the stores must both be [rows, cols, Hkv, D]")
    for name, t in (("k_store", k_store), ("v_store", v_store)):
        if t.dtype != _bf16 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous bf16")
    rows, cols, Hkv, D = shape
    return _rope_append(library().sdpa_rope_append, q, k_new, v_new, (k_store, v_store),
                        (k_store.data_ptr(), v_store.data_ptr()), rows, cols, Hkv, D, seq_info, table, positions,
                        sections, interleaved, window, seg_mode, q_out, status, stream)


def sdpa_rope_append_q4(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, store: Q4Store,
                        seq_info: torch.Tensor, table: torch.Tensor, *, positions: Optional[torch.Tensor] = None,
                        sections: Optional[Sequence[int]] = None, interleaved: bool = False, window: int = 0,
                        seg_mode: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``sdpa_rope_append`` into a 4-bit store, for ``sdpa_varlen_q4``: the rotated keys, rounded to
    bf16, and the values take their 4 bits on the way."""
    rows, cols, Hkv, D, ptrs = _q4(store)
    return _rope_append(library().sdpa_rope_append_fourbit, q, k_new, v_new, store, (ptrs,), rows, cols, Hkv, D,
                        seq_info, table, positions, sections, interleaved, window, seg_mode, q_out, status, stream)


def _unpack(entry, store, store_args, seq_info, T, window, seg_mode, k_out, v_out, status, stream):
    rows, cols, Hkv, D, ptrs = store_args
    seq_ptr, mode_ptr, S = _table(seq_info, seg_mode)
    shape = (T, Hkv, D)
    rs, hs = _strides("k_out", k_out, shape) if k_out is not None else (Hkv * D, D)
    if (_strides("v_out", v_out, shape) if v_out is not None else (Hkv * D, D)) != (rs, hs):
        raise ValueError("k_out and v_out must share strides")
    dev = _device_of(*store, seq_info, seg_mode, k_out, v_out, status)
    if k_out is None:
        k_out = _rows_like(seq_info, shape, stream)
    if v_out is None:
        v_out = _rows_like(seq_info, shape, stream)
    _call(entry, dev, stream, ptrs, rows, cols, Hkv, D, seq_ptr, mode_ptr, S, _window(window), T,
          k_out.data_ptr(), v_out.data_ptr(), rs, hs, _status_ptr(status))
    return k_out, v_out


def sdpa_q4_unpack(store: Q4Store, seq_info: torch.Tensor, T: int, *, window: int = 0,
                   seg_mode: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                   v_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """(k, v) bf16 [T, Hkv, D]: the rows of a segment table as a 4-bit store holds them (exact).
    Row i of a live segment is position kv_end - q_len + i; other rows are 0."""
    return _unpack(library().sdpa_fourbit_unpack, store, _q4(store), seq_info, T, window, seg_mode, k_out, v_out, status,
                   stream)


def q4_workspace_bytes(T: int, Hq: int, store: Q4Store, S: int) -> int:
    """Bytes of workspace ``sdpa_varlen_q4`` needs for these sizes, on the store's device."""
    cols, Hkv, rows, half = store.k_codes.shape
    with torch.cuda.device(store.k_codes.device):
        return int(library().sdpa_varlen_fourbit_workspace_bytes(T, Hq, Hkv, 2 * half, S, rows, cols))


def _attend_packed(entry, workspace_bytes_of, q, store, store_args, seq_info, causal, window, seg_mode, scale, out,
                   workspace, status, stream):
    """Attention over a store of codes, whose checked parts are store_args."""
    rs, hs = _strides("q", q)
    shape = q.shape
    T, Hq, D = shape
    rows, cols, Hkv, Ds, ptrs = store_args
    if Ds != D:
        raise ValueError("head dims of q and the store differ")
    seq_ptr, mode_ptr, S = _table(seq_info, seg_mode)
    ors, ohs = _strides("out", out, shape) if out is not None else (Hq * D, D)
    dev = _device_of(q, *store, seq_info, seg_mode, out, workspace, status)
    if out is None:
        out = _rows_like(q, shape, stream)
    if workspace is None:
        workspace = _workspace(workspace_bytes_of(T, Hq, store, S), q.device, stream)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _call(entry, dev, stream, q.data_ptr(), T, Hq, D, rs, hs, ptrs, rows, cols, Hkv, seq_ptr,
          mode_ptr, S, 1 if causal else 0, _window(window), D ** -0.5 if scale is None else float(scale), out.data_ptr(),
          ors, ohs, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _status_ptr(status))
    return out


def sdpa_varlen_q4(q: torch.Tensor, store: Q4Store, seq_info: torch.Tensor, *, causal: bool, window: int = 0,
                   seg_mode: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``sdpa_varlen`` over a 4-bit store: the attention of the values its codes stand for.
    ``seg_mode`` (int32 [S, 2] (causal, window) per segment) replaces causal and window."""
    return _attend_packed(library().sdpa_varlen_fourbit, q4_workspace_bytes, q, store, _q4(store), seq_info, causal, window,
                          seg_mode, scale, out, workspace, status, stream)


# ------------------------------------------------ the 8-bit column store

class Q8Store(NamedTuple):
    """An 8-bit column store: uint8 codes [cols, Hkv, rows, D] and scales [cols, Hkv, rows / 16] of the
    keys, then of the values; 16 rows of a head share a scale.  Code c under scale byte b stands for
    (c - 128) * 2**(min(b, 29) - 20)."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def q8_store(rows: int, cols: int, Hkv: int, D: int, device=None) -> Q8Store:
    """An empty 8-bit store (every value 0); rows a multiple of 16."""
    if rows <= 0 or rows % 16 or cols <= 0 or Hkv <= 0 or D not in (64, 128, 256):
        raise ValueError("rows must be a multiple of 16, D 64, 128 or 256")
    codes = lambda: torch.full((cols, Hkv, rows, D), 128, dtype=_u8, device=device)  # noqa: E731
    scales = lambda: torch.zeros((cols, Hkv, rows // 16), dtype=_u8, device=device)  # noqa: E731
    return Q8Store(codes(), scales(), codes(), scales())


def _q8(store: Q8Store):
    """(rows, cols, Hkv, D, packed pointers) of an 8-bit store."""
    kc, ks, vc, vs = store
    shape = kc.shape
    if len(shape) != 4 or shape[2] % 16 or vc.shape != shape or ks.shape != vs.shape or \
            ks.shape != (shape[0], shape[1], shape[2] // 16):
        raise ValueError("an 8-bit store is codes [cols, Hkv, rows, D] and scales [cols, Hkv, rows / 16], twice")
    if not (kc.dtype is ks.dtype is vc.dtype is vs.dtype is _u8 and kc.is_contiguous() and ks.is_contiguous() and
            vc.is_contiguous() and vs.is_contiguous()):
        raise ValueError("an 8-bit store's tensors must be contiguous uint8")
    cols, Hkv, rows, D = shape
    return rows, cols, Hkv, D, _Q8_POINTERS.pack(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr())


def sdpa_rope_append_q8(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, store: Q8Store,
                        seq_info: torch.Tensor, table: torch.Tensor, *, positions: Optional[torch.Tensor] = None,
                        sections: Optional[Sequence[int]] = None, interleaved: bool = False, window: int = 0,
                        seg_mode: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``sdpa_rope_append`` into an 8-bit store, for ``sdpa_varlen_q8``: the rotated keys, rounded to
    bf16, and the values take their 8 bits on the way.  Each block of 16 store rows that the step writes to
    gets the smallest scale that holds its new rows and those that hold earlier positions, which are coded
    again where the scale changes.  Segments of one call may share a block of a column: it is coded once, with the
    rows of all of them (a cell that several write takes the last one's)."""
    rows, cols, Hkv, D, ptrs = _q8(store)
    return _rope_append(library().sdpa_rope_append_eightbit, q, k_new, v_new, store, (ptrs,), rows, cols, Hkv, D,
                        seq_info, table, positions, sections, interleaved, window, seg_mode, q_out, status, stream)


def sdpa_q8_unpack(store: Q8Store, seq_info: torch.Tensor, T: int, *, window: int = 0,
                   seg_mode: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                   v_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """(k, v) bf16 [T, Hkv, D]: the rows of a segment table as an 8-bit store holds them (exact).
    Row i of a live segment is position kv_end - q_len + i; other rows are 0."""
    return _unpack(library().sdpa_eightbit_unpack, store, _q8(store), seq_info, T, window, seg_mode, k_out, v_out,
                   status, stream)


def q8_workspace_bytes(T: int, Hq: int, store: Q8Store, S: int) -> int:
    """Bytes of workspace ``sdpa_varlen_q8`` needs for these sizes, on the store's device."""
    cols, Hkv, rows, D = store.k_codes.shape
    with torch.cuda.device(store.k_codes.device):
        return int(library().sdpa_varlen_eightbit_workspace_bytes(T, Hq, Hkv, D, S, rows, cols))


def sdpa_varlen_q8(q: torch.Tensor, store: Q8Store, seq_info: torch.Tensor, *, causal: bool, window: int = 0,
                   seg_mode: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``sdpa_varlen`` over an 8-bit store: the attention of the values its codes stand for.
    ``seg_mode`` (int32 [S, 2] (causal, window) per segment) replaces causal and window."""
    return _attend_packed(library().sdpa_varlen_eightbit, q8_workspace_bytes, q, store, _q8(store), seq_info, causal, window,
                          seg_mode, scale, out, workspace, status, stream)
