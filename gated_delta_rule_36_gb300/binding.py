"""Thin ctypes binding of the KDA C ABI (``include/kda.h``).

Argument marshalling only: every step of the forward runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
CPU fallback: if ``libkda.so`` is missing or the tensors are not on a CUDA device,
the call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import sys
import threading
from typing import Optional

import torch

from . import build as _build

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_ALIAS, KDA_ERR_WORKSPACE, KDA_ERR_CUDA = range(6)
KDA_BF16, KDA_F32, KDA_I64, KDA_U8 = 0, 1, 2, 3
KDA_DEVERR_CU_SEQLENS, KDA_DEVERR_TIMEOUT, KDA_DEVERR_INTERNAL = 0x1, 0x2, 0x4
HEAD_DIM = 128

# Every function include/kda.h declares.
EXPORTED = ("kda_workspace_size", "kda_fwd", "kda_status_string", "kda_last_error",
            "kda_read_device_status", "kda_fwd_no_alloc", "kda_fwd_host_device_bytes", "kda_fwd_host",
            "kda_fwd_host_workspace_offset", "kda_decode", "kda_fwd_ex", "kda_decode_ex", "kda_fwd_schedule",
            "kda_fwd_set_trace", "kda_qk_norm_rope", "kda_attn_workspace_size", "kda_attn_fwd", "kda_lin_workspace_size",
            "kda_lin_fwd", "kda_lin_decode", "kda_qcache_append", "kda_attn_qcache_workspace_size", "kda_attn_qcache_fwd",
            "kda_gated_norm", "kda_residual_norm")
KDA_FLAG_BETA_LOGIT, KDA_FLAG_GATE_SOFTPLUS = 0x1, 0x2
KDA_FLAG_KERNEL_MASK = 0xF00
KDA_KERNEL_DEFAULT, KDA_KERNEL_CHUNK16, KDA_KERNEL_REGISTER_STATE, KDA_KERNEL_BF16_STATE = 0x000, 0x100, 0x200, 0x300
KDA_KERNEL_SMEM_STATE = 0x400
KDA_SCHEDULE_TWO_PER_SM, KDA_SCHEDULE_ONE_PER_SM, KDA_SCHEDULE_CLUSTER, KDA_SCHEDULE_CLUSTER2 = 0, 1, 2, 3
KDA_TRACE_POINTS = 8
KDA_DEVERR_POSITION = 0x8
KDA_FLAG_ROPE_INTERLEAVED = 0x1
KDA_FLAG_GATE_SILU = 0x1
KDA_QCACHE_ROW = 144
KDA_RESIDUAL_MAX_DIM = 16384

_DTYPE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.int64: KDA_I64}


class KdaTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4)]


class KDAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return os.environ.get("KDA_LIBRARY") or _build.LIB_PATH


def load(path: Optional[str] = None):
    """Load libkda.so (raises if it has not been built).  The environment variable
    KDA_LIBRARY names another build of the same ABI to load instead (the tests use it
    for the range-checked build)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or os.environ.get("KDA_LIBRARY") or _build.LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"KDA CUDA library not found at {p}; build it with "
                              "gated_delta_rule_36_gb300.build.build()")
        lib = ctypes.CDLL(p)
        T = ctypes.POINTER(KdaTensor)
        lib.kda_workspace_size.restype = ctypes.c_size_t
        lib.kda_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
        lib.kda_fwd.restype = ctypes.c_int
        lib.kda_fwd.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, ctypes.c_float, T, T, T,
                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [ctypes.c_int]
        lib.kda_last_error.restype = ctypes.c_char_p
        lib.kda_last_error.argtypes = []
        lib.kda_fwd_set_trace.restype = ctypes.c_int
        lib.kda_fwd_set_trace.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64]
        lib.kda_fwd_schedule.restype = ctypes.c_int
        lib.kda_fwd_schedule.argtypes = [ctypes.c_int64, ctypes.c_uint32, ctypes.POINTER(ctypes.c_int32)]
        lib.kda_read_device_status.restype = ctypes.c_int
        lib.kda_read_device_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.POINTER(ctypes.c_uint32)]
        lib.kda_fwd_no_alloc.restype = ctypes.c_int
        lib.kda_fwd_no_alloc.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, ctypes.c_float, T, T, T,
                                         ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]
        lib.kda_fwd_ex.restype = ctypes.c_int
        lib.kda_fwd_ex.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, ctypes.c_float, T, T, T,
                                   ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_void_p]
        lib.kda_decode_ex.restype = ctypes.c_int
        lib.kda_decode_ex.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, ctypes.c_float, T, T,
                                      ctypes.c_uint32, ctypes.c_void_p]
        lib.kda_decode.restype = ctypes.c_int
        lib.kda_decode.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, ctypes.c_float, T, T, ctypes.c_void_p]
        lib.kda_fwd_host_device_bytes.restype = ctypes.c_size_t
        lib.kda_fwd_host_device_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                                                  ctypes.c_int, ctypes.c_int]
        lib.kda_fwd_host_workspace_offset.restype = ctypes.c_size_t
        lib.kda_fwd_host_workspace_offset.argtypes = lib.kda_fwd_host_device_bytes.argtypes
        lib.kda_fwd_host.restype = ctypes.c_int
        lib.kda_fwd_host.argtypes = [T, T, T, T, T, ctypes.c_float, T, T, T, ctypes.c_float, T, T, T,
                                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p]
        D, V, F = ctypes.c_char_p, ctypes.c_void_p, ctypes.c_float   # D: a packed kda_view or kda_tensor (_view, _dense)
        lib.kda_qk_norm_rope.restype = ctypes.c_int
        lib.kda_qk_norm_rope.argtypes = [D, D, D, D, F, D, D, D, D, V, ctypes.c_uint32, V]
        lib.kda_attn_workspace_size.restype = ctypes.c_size_t
        lib.kda_attn_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
        lib.kda_attn_fwd.restype = ctypes.c_int
        lib.kda_attn_fwd.argtypes = [D, D, D, F, D, D, D, D, D, V, ctypes.c_size_t, V]
        lib.kda_lin_workspace_size.restype = ctypes.c_size_t
        lib.kda_lin_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int]
        lib.kda_lin_fwd.restype = ctypes.c_int
        lib.kda_lin_fwd.argtypes = [D, D, D, D, F, D, D, D, D, V, ctypes.c_size_t, V]
        lib.kda_lin_decode.restype = ctypes.c_int
        lib.kda_lin_decode.argtypes = [D, D, D, D, F, D, D, D, V]
        lib.kda_qcache_append.restype = ctypes.c_int
        lib.kda_qcache_append.argtypes = [D, D, D, D, D, D, D, V, V]
        lib.kda_attn_qcache_workspace_size.restype = ctypes.c_size_t
        lib.kda_attn_qcache_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
        lib.kda_attn_qcache_fwd.restype = ctypes.c_int
        lib.kda_attn_qcache_fwd.argtypes = [D, D, F, D, D, D, D, V, ctypes.c_size_t, V]
        lib.kda_gated_norm.restype = ctypes.c_int
        lib.kda_gated_norm.argtypes = [D, D, D, D, F, ctypes.c_uint32, V]
        lib.kda_residual_norm.restype = ctypes.c_int
        lib.kda_residual_norm.argtypes = [D, D, D, D, F, D, D, D, F, V]
        if path is None:
            _lib = lib
        return lib


def _desc(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (the KDA path has no CPU fallback)")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.dim() > 4:
        raise ValueError(f"{name}: at most 4 dims")
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    d = KdaTensor()
    d.data = t.data_ptr() if t.numel() > 0 else (t.data_ptr() or 16)
    d.dtype = _DTYPE[t.dtype]
    d.ndim = t.dim()
    for i, s in enumerate(t.shape):
        d.shape[i] = int(s)
    return d


def _hdesc(t: Optional[torch.Tensor], name: str):
    """Descriptor of a host (CPU) tensor for kda_fwd_host."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name}: kda_fwd_host takes host tensors")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.dim() > 4 or t.dtype not in _DTYPE:
        raise ValueError(f"{name}: unsupported shape or dtype")
    d = KdaTensor()
    d.data = t.data_ptr() if t.numel() > 0 else (t.data_ptr() or 16)
    d.dtype = _DTYPE[t.dtype]
    d.ndim = t.dim()
    for i, s in enumerate(t.shape):
        d.shape[i] = int(s)
    return d


def _state_code(t):
    return -1 if t is None else _DTYPE[t.dtype]


def kda_fwd_host_device_bytes(q, cu_seqlens=None, initial_state=None, final_state=None) -> int:
    """Device bytes kda_fwd_host needs for these (host) tensors."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    N = (cu_seqlens.shape[0] - 1) if cu_seqlens is not None else 0
    return int(load().kda_fwd_host_device_bytes(B, T, H, N, _state_code(initial_state), _state_code(final_state)))


def kda_fwd_host_workspace_offset(q, cu_seqlens=None, initial_state=None, final_state=None) -> int:
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    N = (cu_seqlens.shape[0] - 1) if cu_seqlens is not None else 0
    return int(load().kda_fwd_host_workspace_offset(B, T, H, N, _state_code(initial_state),
                                                    _state_code(final_state)))


def kda_fwd_host(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, initial_state=None,
                 final_state=None, cu_seqlens=None, device_buffer=None, groups=0, stream=None):
    """The forward on host tensors (pinned for asynchronous copies): copies in, computes
    and copies ``out`` / ``final_state`` back, pipelined over groups of sequences.
    ``device_buffer`` is a uint8 CUDA tensor of at least kda_fwd_host_device_bytes bytes.
    Returns once the work is enqueued on ``stream`` (torch's current stream by default)."""
    lib = load()
    descs = [_hdesc(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (out, "out"),
                                       (A_log, "A_log"), (dt_bias, "dt_bias"), (initial_state, "initial_state"),
                                       (final_state, "final_state"), (cu_seqlens, "cu_seqlens"))]
    dq, dk, dv, dg, db, do, da, dd, di, df, dc = descs
    if device_buffer is None or not (isinstance(device_buffer, torch.Tensor) and device_buffer.is_cuda
                                     and device_buffer.dtype == torch.uint8):
        raise ValueError("device_buffer: must be a uint8 CUDA tensor")
    if stream is None:
        stream = torch.cuda.current_stream(device_buffer.device)
    sh = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    st = lib.kda_fwd_host(_ref(dq), _ref(dk), _ref(dv), _ref(dg), _ref(db), ctypes.c_float(float(scale)),
                          _ref(do), _ref(da), _ref(dd), ctypes.c_float(float(lower_bound)), _ref(di),
                          _ref(df), _ref(dc), ctypes.c_void_p(device_buffer.data_ptr()),
                          ctypes.c_size_t(device_buffer.numel()), ctypes.c_int(int(groups)), ctypes.c_void_p(sh))
    _check(lib, st)
    return device_buffer


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _check(lib, st: int):
    if st != KDA_OK:
        detail = lib.kda_last_error().decode()
        raise KDAError(st, f"{lib.kda_status_string(st).decode()}: {detail}")


def kda_workspace_size(T_total: int, H: int, N: int) -> int:
    return int(load().kda_workspace_size(int(T_total), int(H), int(N)))


def kda_fwd(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, initial_state=None,
            final_state=None, cu_seqlens=None, workspace=None, stream=None, flags=0):
    """Run the forward through the C ABI.  Tensors as in ``include/kda.h``.

    ``workspace`` (uint8 CUDA tensor) is allocated with torch when omitted;
    ``stream`` defaults to torch's current stream of q's device; ``flags`` (KDA_FLAG_*
    bits, plus one KDA_KERNEL_* value) selects the interface variants and the kernel
    through kda_fwd_ex.  Returns the workspace (its
    first word is the device status).
    """
    lib = load()
    descs = [_desc(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (out, "out"),
                                      (A_log, "A_log"), (dt_bias, "dt_bias"), (initial_state, "initial_state"),
                                      (final_state, "final_state"), (cu_seqlens, "cu_seqlens"))]
    dq, dk, dv, dg, db, do, da, dd, di, df, dc = descs
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    nseq = (cu_seqlens.shape[0] - 1) if cu_seqlens is not None else B
    if workspace is None:
        workspace = torch.empty(kda_workspace_size(B * T, H, nseq), dtype=torch.uint8, device=q.device)
    if not (workspace.is_cuda and workspace.dtype == torch.uint8):
        raise ValueError("workspace: must be a uint8 CUDA tensor")
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sh = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    args = (_ref(dq), _ref(dk), _ref(dv), _ref(dg), _ref(db), ctypes.c_float(float(scale)),
            _ref(do), _ref(da), _ref(dd), ctypes.c_float(float(lower_bound)), _ref(di),
            _ref(df), _ref(dc), ctypes.c_void_p(workspace.data_ptr()), ctypes.c_size_t(workspace.numel()))
    if flags:
        st = lib.kda_fwd_ex(*args, ctypes.c_uint32(int(flags)), ctypes.c_void_p(sh))
    else:
        st = lib.kda_fwd(*args, ctypes.c_void_p(sh))
    _check(lib, st)
    return workspace


def kda_decode(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, initial_state=None, final_state=None,
               stream=None, flags=0):
    """One decode step (one token per sequence) through the C ABI: q, k, v, g, out
    [B, H, 128], beta [B, H], states [B, H, 128, 128]; final_state may be initial_state
    itself for the in-place update."""
    lib = load()
    descs = [_desc(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (out, "out"),
                                      (A_log, "A_log"), (dt_bias, "dt_bias"), (initial_state, "initial_state"),
                                      (final_state, "final_state"))]
    dq, dk, dv, dg, db, do, da, dd, di, df = descs
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sh = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    args = (_ref(dq), _ref(dk), _ref(dv), _ref(dg), _ref(db), ctypes.c_float(float(scale)), _ref(do),
            _ref(da), _ref(dd), ctypes.c_float(float(lower_bound)), _ref(di), _ref(df))
    if flags:
        st = lib.kda_decode_ex(*args, ctypes.c_uint32(int(flags)), ctypes.c_void_p(sh))
    else:
        st = lib.kda_decode(*args, ctypes.c_void_p(sh))
    _check(lib, st)


def kda_fwd_set_trace(buffer=None, unit: int = 0) -> None:
    """Record the chain trace of (sequence, head) unit ``unit`` (sequence * H + head) into
    ``buffer`` (a CUDA int64 tensor of [chunks, KDA_TRACE_POINTS]) on later forward launches
    of this thread that take the cluster schedule; ``None`` turns it off."""
    lib = load()
    if buffer is None:
        _check(lib, lib.kda_fwd_set_trace(None, 0, 0))
        return
    if not (isinstance(buffer, torch.Tensor) and buffer.is_cuda and buffer.is_contiguous()):
        raise KDAError(KDA_ERR_INVALID_ARG, "trace buffer must be a contiguous CUDA tensor")
    _check(lib, lib.kda_fwd_set_trace(ctypes.c_void_p(buffer.data_ptr()), buffer.numel() * buffer.element_size(),
                                      int(unit)))


def kda_fwd_schedule(units: int, flags: int = 0) -> int:
    """KDA_SCHEDULE_* that kda_fwd takes on the current device for ``units`` (sequence, head)
    units: two CTAs per SM, one CTA per SM, or a cluster of four or of two CTAs per unit."""
    lib = load()
    sched = ctypes.c_int32(-1)
    _check(lib, lib.kda_fwd_schedule(int(units), int(flags), ctypes.byref(sched)))
    return int(sched.value)


def kda_read_device_status(workspace, stream=None) -> int:
    """Status bits of the last call that used ``workspace`` (a uint8 CUDA tensor, or
    the device address kda_fwd_no_alloc returns).  Synchronises the stream."""
    lib = load()
    if isinstance(workspace, torch.Tensor):
        addr, device = workspace.data_ptr(), workspace.device
    else:
        addr, device = int(workspace), torch.device("cuda", torch.cuda.current_device())
    if stream is None:
        stream = torch.cuda.current_stream(device)
    sh = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    bits = ctypes.c_uint32(0)
    _check(lib, lib.kda_read_device_status(ctypes.c_void_p(addr), ctypes.c_void_p(sh), ctypes.byref(bits)))
    return int(bits.value)


def kda_fwd_no_alloc(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, initial_state=None,
                     final_state=None, cu_seqlens=None, stream=None) -> int:
    """kda_fwd for callers that cannot allocate device memory: the library uses its
    own fixed device array (KDA_NO_ALLOC_MAX_SEQS sequences at most) as the workspace
    and nothing is allocated.  Calls that overlap on the GPU share that array and
    race.  Returns the array's device address (for kda_read_device_status)."""
    lib = load()
    descs = [_desc(t, n) for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (out, "out"),
                                      (A_log, "A_log"), (dt_bias, "dt_bias"), (initial_state, "initial_state"),
                                      (final_state, "final_state"), (cu_seqlens, "cu_seqlens"))]
    dq, dk, dv, dg, db, do, da, dd, di, df, dc = descs
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    sh = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    used = ctypes.c_void_p(0)
    st = lib.kda_fwd_no_alloc(_ref(dq), _ref(dk), _ref(dv), _ref(dg), _ref(db), ctypes.c_float(float(scale)),
                              _ref(do), _ref(da), _ref(dd), ctypes.c_float(float(lower_bound)), _ref(di),
                              _ref(df), _ref(dc), ctypes.c_void_p(sh), ctypes.byref(used))
    _check(lib, st)
    return int(used.value or 0)


def fwd(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, initial_state=None,
        final_state=None, cu_seqlens=None):
    """FlashKDA-style convenience call: allocates the workspace, writes ``out`` and
    ``final_state`` in place and returns ``out``."""
    kda_fwd(q, k, v, g, beta, scale, out, A_log, dt_bias, lower_bound, initial_state=initial_state,
            final_state=final_state, cu_seqlens=cu_seqlens)
    return out


# ---------------------------------------------------------------------------
# The token mixers beside KDA.  Their small calls last a few microseconds on the GPU, so the
# descriptors are packed straight into bytes (the layout of kda_view, whose first 48 bytes are
# a kda_tensor) instead of filling ctypes structures field by field.
# ---------------------------------------------------------------------------
_PACK_VIEW = struct.Struct("=Qii4q4q").pack
_PACK_VIEW2, _PACK_VIEW3 = struct.Struct("=Qii2q16x2q16x").pack, struct.Struct("=Qii3q8x3q8x").pack   # (0.2 us less than the former)
_PACK_DENSE, _PACK_DENSE1 = struct.Struct("=Qii4q").pack, struct.Struct("=Qiiq24x").pack
_PAD = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())


def _bad_tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (there is no CPU fallback)")
    if t.dim() > 4:
        raise ValueError(f"{name}: at most 4 dims")
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    raise ValueError(f"{name}: on another device than the first tensor")


def _view(t, name, device):
    """The packed kda_view of a CUDA tensor of any strides."""
    if t is None:
        return None
    dtype = _DTYPE.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dtype is None or t.get_device() != device or device < 0:
        _bad_tensor(t, name)
    shape = t.shape
    n = len(shape)
    if n == 3:
        a, b, c = shape
        x, y, z = t.stride()
        return _PACK_VIEW3(t.data_ptr() or 16, dtype, 3, a, b, c, x, y, z)
    if n == 2:
        a, b = shape
        x, y = t.stride()
        return _PACK_VIEW2(t.data_ptr() or 16, dtype, 2, a, b, x, y)
    if n > 4:
        _bad_tensor(t, name)
    pad = _PAD[n]
    return _PACK_VIEW(t.data_ptr() or 16, dtype, n, *shape, *pad, *t.stride(), *pad)


def _bytes_view(t, name, device):
    """The packed kda_view of a uint8 CUDA tensor of any strides (a cache in 4 bits)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != torch.uint8 or t.get_device() != device or device < 0 or t.dim() != 4:
        raise ValueError(f"{name}: must be a uint8 CUDA tensor [N, S, Hk, {KDA_QCACHE_ROW}] on the other tensors' device")
    n, s, h, b = t.shape
    sn, ss, sh, sb = t.stride()
    return _PACK_VIEW(t.data_ptr() or 16, KDA_U8, 4, n, s, h, b, sn, ss, sh, sb)


def _status_word(status, device):
    if status is None:
        return None
    if not (isinstance(status, torch.Tensor) and status.get_device() == device and status.dtype == torch.uint8 and status.numel() >= 4):
        raise ValueError("status: must be a uint8 CUDA tensor of at least 4 bytes on the other tensors' device")
    return status.data_ptr()


def _dense(t, name, device):
    """The packed kda_tensor of a contiguous CUDA tensor."""
    if t is None:
        return None
    dtype = _DTYPE.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dtype is None or t.get_device() != device or device < 0:
        _bad_tensor(t, name)
    shape = t.shape
    n = len(shape)
    if n > 4:
        _bad_tensor(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if n == 1:
        return _PACK_DENSE1(t.data_ptr() or 16, dtype, 1, shape[0])
    return _PACK_DENSE(t.data_ptr() or 16, dtype, n, *shape, *_PAD[n])


def _device(t, name):
    """The device of a call: the first tensor's, which has to be the current one (the kernels go there)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    device = t.get_device()
    if device >= 0 and device != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on cuda:{device}, which is not the current device")
    return device


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)   # (a Stream object would cost a microsecond)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _workspace(workspace, nbytes, device, stream):
    """The caller's workspace, or one from torch that belongs to ``stream``: neither what its memory held
    before nor what it holds after the call is in use on another stream."""
    if workspace is None:
        if stream is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream, device), device=device)
        with torch.cuda.stream(stream):
            return torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
    elif not (isinstance(workspace, torch.Tensor) and workspace.get_device() == device and workspace.dtype == torch.uint8
              and workspace.is_contiguous()):
        raise ValueError("workspace: must be a contiguous uint8 CUDA tensor on the other tensors' device")
    return workspace


# Workspaces of attention over a 4-bit cache: an allocation between two launches costs 8 us of host time, more than the
# rest of the call, so the last one of every stream is kept (if it is small) and taken again once nobody else holds it.
# Of so many streams at most: those of streams that are no more go with the others then.
_KEPT, _KEPT_MOST, _KEPT_STREAMS = {}, 32 << 20, 32
_storage_uses = getattr(torch._C, "_storage_Use_Count", None)
_refs = sys.getrefcount


def _kept_and_uses(kept):
    """A kept workspace, which the caller holds from here on, and the references that there are to it and its storage (views
    hold the storage).  How many of them are the interpreter's and torch's own differs between versions."""
    ws, storage, handle = kept[0], kept[1], kept[4]
    return ws, (_refs(ws), _refs(storage), _storage_uses(handle))


def _to_keep(nbytes, device):
    ws = _workspace(None, nbytes, device, None)
    storage = ws.untyped_storage()
    _storage_uses(storage._cdata)   # (asking once may make an object that stays)
    return [ws, storage, ws.data_ptr(), nbytes, storage._cdata, None]


def _kept_workspace(nbytes, device, stream, raw):
    """A workspace from torch for a call on ``stream`` (``raw``: its handle), and where it is.  On the current stream it is
    that of the stream's call before, if neither the caller nor a view keeps it: what it held is used by earlier work of that
    stream only.  Calls that are captured into a graph get their own, as memory of the graph."""
    if stream is not None or nbytes > _KEPT_MOST or _storage_uses is None or torch._C._cuda_isCurrentStreamCapturing():
        ws = _workspace(None, nbytes, device, stream)
        return ws, ws.data_ptr(), ws.numel()
    kept = _KEPT.get((device, raw))
    if kept is not None and kept[3] >= nbytes:
        ws, uses = _kept_and_uses(kept)
        if uses == kept[5]:
            return ws, kept[2], kept[3]
        del ws
    kept = _to_keep(nbytes, device)
    ws, kept[5] = _kept_and_uses(kept)   # (nobody else holds it yet)
    if len(_KEPT) >= _KEPT_STREAMS and (device, raw) not in _KEPT:
        _KEPT.clear()
    _KEPT[device, raw] = kept
    return ws, kept[2], nbytes


def kda_qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, eps=1e-6, status=None, flags=0,
                     stream=None):
    """RMS norm of every head of q [T, Hq, 128] and k [T, Hk, 128] and the rotary rotation, in
    one pass; q_out / k_out may be q / k themselves.  Tensors as in ``include/kda.h``; q and k
    may be strided views of one projection buffer.  ``status``: a CUDA uint8 tensor of at least 4
    bytes whose first word collects KDA_DEVERR_POSITION (see kda_read_device_status)."""
    lib = _lib or load()
    dev = _device(q, "q")
    if status is not None and not (isinstance(status, torch.Tensor) and status.get_device() == dev
                                   and status.dtype == torch.uint8 and status.numel() >= 4):
        raise ValueError("status: must be a uint8 CUDA tensor of at least 4 bytes on the other tensors' device")
    st = lib.kda_qk_norm_rope(_view(q, "q", dev), _view(k, "k", dev), _dense(q_weight, "q_weight", dev),
                              _dense(k_weight, "k_weight", dev), eps, _dense(cos_sin, "cos_sin", dev),
                              _dense(positions, "positions", dev), _view(q_out, "q_out", dev), _view(k_out, "k_out", dev),
                              None if status is None else status.data_ptr(), flags, _stream(stream, dev))
    if st:
        _check(lib, st)


def kda_attn_workspace_size(Tq: int, Hq: int, Hk: int) -> int:
    return int(load().kda_attn_workspace_size(int(Tq), int(Hq), int(Hk)))


def kda_attn_fwd(q, k, v, scale, out, lse=None, cu_seqlens_q=None, cu_seqlens_k=None, seqlens_k=None, workspace=None,
                 stream=None):
    """Causal softmax attention with grouped heads: q, out [Tq, Hq, 128]; k, v [Tk, Hk, 128]
    (packed prompts) or [N, S, Hk, 128] with ``seqlens_k`` (caches; one or more new tokens per
    sequence).  Tensors and modes as in ``include/kda.h``.  ``workspace`` (uint8 CUDA tensor) is
    allocated with torch when omitted.  Returns the workspace (its first word is the device status)."""
    lib = _lib or load()
    dev = _device(q, "q")
    dq, dk = _view(q, "q", dev), _view(k, "k", dev)
    if workspace is None and q.dim() == 3 and k is not None and k.dim() in (3, 4):
        nbytes = lib.kda_attn_workspace_size(q.shape[0], q.shape[1], k.shape[-2]) or 256   # 0: refused below
        workspace = _workspace(None, nbytes, dev, stream)
    else:
        workspace = _workspace(workspace, 256, dev, stream)
    st = lib.kda_attn_fwd(dq, dk, _view(v, "v", dev), scale, _view(out, "out", dev), _dense(lse, "lse", dev),
                          _dense(cu_seqlens_q, "cu_seqlens_q", dev), _dense(cu_seqlens_k, "cu_seqlens_k", dev),
                          _dense(seqlens_k, "seqlens_k", dev), workspace.data_ptr(), workspace.numel(),
                          _stream(stream, dev))
    if st:
        _check(lib, st)
    return workspace


def kda_lin_workspace_size(T_total: int, H: int, N: int) -> int:
    return int(load().kda_lin_workspace_size(int(T_total), int(H), int(N)))


def kda_lin_fwd(q, k, v, log_decay, scale, out, initial_state=None, final_state=None, cu_seqlens=None, workspace=None,
                stream=None):
    """Linear attention with a decay for each head over prompts: q, k, v, out [B, T, H, 128],
    log_decay [H], states [Nseq, H, 128, 128]; packed with ``cu_seqlens`` as kda_fwd.  Tensors as in
    ``include/kda.h``.  Returns the workspace (its first word is the device status)."""
    lib = _lib or load()
    dev = _device(q, "q")
    dq = _view(q, "q", dev)
    if workspace is None and q.dim() == 4:
        B, T, H, _ = q.shape
        nseq = B if cu_seqlens is None else max(cu_seqlens.numel() - 1, 0)
        workspace = _workspace(None, lib.kda_lin_workspace_size(B * T, H, nseq), dev, stream)
    else:
        workspace = _workspace(workspace, 256, dev, stream)
    st = lib.kda_lin_fwd(dq, _view(k, "k", dev), _view(v, "v", dev), _dense(log_decay, "log_decay", dev), scale,
                         _view(out, "out", dev), _dense(initial_state, "initial_state", dev),
                         _dense(final_state, "final_state", dev), _dense(cu_seqlens, "cu_seqlens", dev),
                         workspace.data_ptr(), workspace.numel(), _stream(stream, dev))
    if st:
        _check(lib, st)
    return workspace


def kda_lin_decode(q, k, v, log_decay, scale, out, initial_state=None, final_state=None, stream=None):
    """One token of kda_lin_fwd's recurrence for every sequence: q, k, v, out [B, H, 128],
    states [B, H, 128, 128]; final_state may be initial_state itself."""
    lib = _lib or load()
    dev = _device(q, "q")
    st = lib.kda_lin_decode(_view(q, "q", dev), _view(k, "k", dev), _view(v, "v", dev),
                            _dense(log_decay, "log_decay", dev), scale, _view(out, "out", dev),
                            _dense(initial_state, "initial_state", dev), _dense(final_state, "final_state", dev),
                            _stream(stream, dev))
    if st:
        _check(lib, st)


# ---------------------------------------------------------------------------
# Around the mixers: a cache in 4 bits and the attention over it, and the norms between the blocks.
# ---------------------------------------------------------------------------
def kda_qcache_append(k, v, cache, seqlens_k, cu_seqlens=None, k_out=None, v_out=None, status=None, stream=None):
    """Append keys and values k, v [T, Hk, 128] to a cache in 4 bits, uint8 [N, S, Hk, KDA_QCACHE_ROW]: sequence n's
    new tokens end at position seqlens_k[n].  ``k_out`` / ``v_out`` (may be k / v themselves) receive the
    values that the cache now stands for.  ``status``: a CUDA uint8 tensor of at least 4 bytes whose first word
    collects KDA_DEVERR_CU_SEQLENS (see kda_read_device_status).  Tensors as in ``include/kda.h``."""
    lib = _lib or load()
    dev = _device(k, "k")
    dc, word = _bytes_view(cache, "cache", dev), _status_word(status, dev)
    st = lib.kda_qcache_append(_view(k, "k", dev), _view(v, "v", dev), dc, _dense(seqlens_k, "seqlens_k", dev),
                               _dense(cu_seqlens, "cu_seqlens", dev), _view(k_out, "k_out", dev), _view(v_out, "v_out", dev), word,
                               _stream(stream, dev))
    if st:
        _check(lib, st)


def kda_attn_qcache_workspace_size(Tq: int, Hq: int, Hk: int, N: int, S: int) -> int:
    return int(load().kda_attn_qcache_workspace_size(int(Tq), int(Hq), int(Hk), int(N), int(S)))


_QCACHE_SIZES = {}   # (Tq, Hq, Hk, N, S): bytes


def kda_attn_qcache_fwd(q, cache, scale, out, seqlens_k, lse=None, cu_seqlens_q=None, workspace=None, stream=None):
    """Causal softmax attention with grouped heads over a cache in 4 bits: q, out [Tq, Hq, 128], cache uint8
    [N, S, Hk, KDA_QCACHE_ROW], seqlens_k [N].  Modes as kda_attn_fwd's over a cache, tensors as in
    ``include/kda.h``.  Returns the workspace (its first word is the device status); one that is allocated here
    serves the stream's next such call once it is dropped."""
    lib = _lib or load()
    dev = _device(q, "q")
    dq, dc, raw = _view(q, "q", dev), _bytes_view(cache, "cache", dev), _stream(stream, dev)
    if workspace is None and q.dim() == 3:
        nseq, S, Hk, _ = cache.shape
        Tq, Hq, _ = q.shape
        sizes = (Tq, Hq, Hk, nseq if cu_seqlens_q is None else max(cu_seqlens_q.numel() - 1, 0), S)
        nbytes = _QCACHE_SIZES.get(sizes)
        if nbytes is None:
            if len(_QCACHE_SIZES) > 4096:
                _QCACHE_SIZES.clear()
            nbytes = _QCACHE_SIZES[sizes] = lib.kda_attn_qcache_workspace_size(*sizes) or 256   # 0: refused below
        workspace, at, room = _kept_workspace(nbytes, dev, stream, raw)
    else:
        workspace = _workspace(workspace, 256, dev, stream)
        at, room = workspace.data_ptr(), workspace.numel()
    st = lib.kda_attn_qcache_fwd(dq, dc, scale, _view(out, "out", dev), _dense(seqlens_k, "seqlens_k", dev), _dense(lse, "lse", dev),
                                 _dense(cu_seqlens_q, "cu_seqlens_q", dev), at, room, raw)
    if st:
        _check(lib, st)
    return workspace


def kda_gated_norm(x, gate, weight, out, eps=1e-6, flags=0, stream=None):
    """RMS norm of every head of x [T, H, 128] times sigmoid(gate) (g sigmoid(g) with KDA_FLAG_GATE_SILU); out may be
    x or gate itself.  Tensors as in ``include/kda.h``; all may be strided views."""
    lib = _lib or load()
    dev = _device(x, "x")
    st = lib.kda_gated_norm(_view(x, "x", dev), _view(gate, "gate", dev), _dense(weight, "weight", dev), _view(out, "out", dev), eps,
                            flags, _stream(stream, dev))
    if st:
        _check(lib, st)


def kda_residual_norm(y, residual, pre_weight, out, residual_out=None, post_weight=None, gate=None, scale=1.0, eps=1e-6, stream=None):
    """r = residual + scale * gate * norm(y) (the norm with ``post_weight``, the gate if given) into ``residual_out``, and
    norm(r) * pre_weight into ``out``: y, out bf16 [T, D], the stream bf16 or fp32.  With y None: the norm of the
    stream alone.  Tensors as in ``include/kda.h``."""
    lib = _lib or load()
    dev = _device(residual, "residual")
    st = lib.kda_residual_norm(_view(y, "y", dev), _view(residual, "residual", dev), _dense(post_weight, "post_weight", dev),
                               _view(gate, "gate", dev), scale, _dense(pre_weight, "pre_weight", dev),
                               _view(residual_out, "residual_out", dev), _view(out, "out", dev), eps, _stream(stream, dev))
    if st:
        _check(lib, st)
