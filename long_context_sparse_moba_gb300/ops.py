"""Python binding of ``libmoba_gb300.so`` (argument marshalling only).

Every function below calls the C ABI of ``include/moba.h`` with the tensors'
device pointers and the current CUDA stream; all arithmetic runs in the
library's kernels.  There is no fallback: if the library is missing or a call
fails, a ``RuntimeError`` is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoba_gb300.so")

MOBA_OK = 0
MOBA_ERR_INVALID_ARG = 1
MOBA_ERR_UNSUPPORTED = 2
MOBA_ERR_CUDA = 3
MOBA_ERR_WORKSPACE = 4
MOBA_ERR_TIMEOUT = 5

_lib = None

_P, _I, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_F, _DB, _LL = ctypes.c_float, ctypes.c_double, ctypes.c_longlong
_SIGNATURES = {
    "moba_num_blocks": (_I, [_I, _I]),
    "moba_status_string": (ctypes.c_char_p, [_I]),
    "moba_last_cuda_error": (ctypes.c_char_p, []),
    "moba_kpool": (_I, [_P, _P, _I, _I, _I, _I, _I, _P]),
    "moba_kpool_varlen": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "moba_gate_topk": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_gate_topk_varlen": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_attn_fwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moba_attn_fwd_ws": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "moba_attn_fwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    "moba_attn_fwd_varlen_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "moba_attn_fwd_varlen_ws": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                     _P, _SZ, _P]),
    "moba_get_status": (_I, [_P]),
    "moba_launch_count": (ctypes.c_ulonglong, []),
    "moba_decode_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_decode_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "moba_decode_fwd_ws": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ,
                                _P]),
    "moba_attn_fwd_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_attn_fwd_noalloc_capacity": (_SZ, []),
    "moba_debug_timeout_info": (None, [_P]),
    "moba_attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_attn_bwd_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moba_attn_bwd_ws": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P,
                              _SZ, _P]),
    "moba_attn_bwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I,
                                  _I, _I, _P]),
    "moba_attn_bwd_varlen_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "moba_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moba_kpool_ex": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "moba_kpool_varlen_ex": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "moba_gate_topk_ex": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "moba_gate_topk_varlen_ex": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "moba_attn_fwd_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moba_attn_fwd_host": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moba_attn_fwd_host_scratch_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moba_attn_fwd_varlen_ex": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                                     _P, _SZ, _P]),
    "moba_attn_bwd_ex": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P,
                              _P, _SZ, _P]),
    "moba_rope": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _LL, _LL, _LL, _LL, _P]),
    "moba_rope_bwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _LL, _LL, _LL, _LL,
                           _P]),
    "moba_rope_frequencies": (_I, [_P, _I, _DB, _I, _DB, _DB, _DB, _DB]),
    "moba_paged_append": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                               _P, _P]),
    "moba_paged_attn": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                             _I, _I, _I, _P, _SZ, _P]),
    "moba_paged_attn_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "moba_page_copy": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "moba_attn_bwd_varlen_ex": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                     _I, _I, _I, _P, _P, _SZ, _P]),
}

POOL_MEAN = 0
POOL_MAX = 1
GATE_TCGEN05 = 0
GATE_CUDA_CORES = 1
ATTN_TCGEN05 = 0
ATTN_MMA_SYNC = 1
SCHEDULE_ADAPTIVE = 0
SCHEDULE_BLOCK_MAJOR = 1


class Options(ctypes.Structure):
    """``moba_options_t``: per-call options (all zero = the defaults)."""
    _fields_ = [("pooling", ctypes.c_int), ("gate_kernel", ctypes.c_int),
                ("attn_kernel", ctypes.c_int), ("debug_flags", ctypes.c_int),
                ("wait_limit_cycles", ctypes.c_longlong), ("idx_out", ctypes.c_void_p),
                ("phase_events", ctypes.c_void_p), ("schedule", ctypes.c_int),
                ("idx_in", ctypes.c_void_p)]


def _options(pooling=POOL_MEAN, gate_kernel=GATE_TCGEN05, attn_kernel=ATTN_TCGEN05,
             debug_flags=0, wait_limit_cycles=0, idx_out=None, phase_events=None,
             schedule=SCHEDULE_ADAPTIVE, idx_in=None):
    """An Options structure and the objects that must outlive the call."""
    o = Options(int(pooling), int(gate_kernel), int(attn_kernel), int(debug_flags),
                int(wait_limit_cycles), None, None, int(schedule), None)
    keep = []
    if idx_out is not None:
        o.idx_out = idx_out.data_ptr()
    if idx_in is not None:
        if idx_in.dtype != torch.int32 or not idx_in.is_cuda or not idx_in.is_contiguous():
            raise ValueError("idx_in must be a contiguous int32 CUDA tensor")
        o.idx_in = idx_in.data_ptr()
    if phase_events is not None:
        if len(phase_events) != len(PHASES) + 1:
            raise ValueError(f"phase_events needs {len(PHASES) + 1} events")
        arr = (ctypes.c_void_p * len(phase_events))()
        for i, ev in enumerate(phase_events):
            arr[i] = ev.cuda_event
        o.phase_events = ctypes.cast(arr, ctypes.c_void_p)
        keep.append(arr)
    return o, keep

PHASES = ("tables", "kpool", "gate", "regroup", "attn_past", "attn_current")


def phase_events(stream=None):
    """Seven timing events for the forward's ``phase_events`` option, created on
    the stream (torch creates an event's CUDA handle at its first record)."""
    st = stream if stream is not None else torch.cuda.current_stream()
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(len(PHASES) + 1)]
    for e in evs:
        e.record(st)
    return evs


def phase_ms(events) -> dict:
    """{phase: ms} between the recorded events (synchronises the last one)."""
    events[-1].synchronize()
    return {name: events[i].elapsed_time(events[i + 1]) for i, name in enumerate(PHASES)}


def lib():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m long_context_sparse_moba_gb300.build` (needs nvcc)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(code: int) -> str:
    return lib().moba_status_string(code).decode()


def _check(code: int, what: str):
    if code != MOBA_OK:
        extra = ""
        if code == MOBA_ERR_CUDA:
            extra = ": " + lib().moba_last_cuda_error().decode()
        raise RuntimeError(f"{what} failed: {status_string(code)} ({code}){extra}")


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, name):
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _out(t, shape, dtype, like, name):
    """A result buffer: a new tensor on like's device, or the caller's one
    after checking its dtype, layout, shape and device."""
    shape = tuple(int(x) for x in shape)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _need(t, dtype, name)
    if tuple(t.shape) != shape or t.device != like.device:
        raise ValueError(f"{name} must have shape {shape} on {like.device}")
    return t


def _ws(workspace):
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    return workspace


def num_blocks(length: int, block_size: int) -> int:
    return int(lib().moba_num_blocks(int(length), int(block_size)))


def _nb_total(cu_host, block_size):
    return sum(num_blocks(cu_host[b + 1] - cu_host[b], block_size) for b in range(len(cu_host) - 1))


def kpool(k, block_size: int, stream=None, pooling=POOL_MEAN):
    """Pooled keys of k [B, S, H, D] -> kbar [B * n, H, D] fp32 (mean, or the
    element-wise maximum with ``pooling=POOL_MAX``)."""
    _need(k, torch.bfloat16, "k")
    B, S, H, D = k.shape
    kbar = torch.empty(B * num_blocks(S, block_size), H, D, dtype=torch.float32, device=k.device)
    o, _keep = _options(pooling=pooling)
    _check(lib().moba_kpool_ex(_ptr(k), _ptr(kbar), B, H, S, D, block_size, ctypes.byref(o),
                               _stream(stream)), "moba_kpool")
    return kbar


def kpool_varlen(k, cu_seqlens, block_size: int, stream=None, pooling=POOL_MEAN):
    """Varlen k [total, H, D], cu_seqlens int32 CUDA [num_seqs + 1]."""
    _need(k, torch.bfloat16, "k")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    total, H, D = k.shape
    nb = _nb_total(cu_seqlens.tolist(), block_size)
    kbar = torch.empty(nb, H, D, dtype=torch.float32, device=k.device)
    o, _keep = _options(pooling=pooling)
    _check(lib().moba_kpool_varlen_ex(_ptr(k), _ptr(kbar), _ptr(cu_seqlens),
                                      cu_seqlens.numel() - 1, total, H, D, block_size,
                                      ctypes.byref(o), _stream(stream)), "moba_kpool_varlen")
    return kbar


def gate_topk(q, kbar, block_size: int, topk: int, stream=None, gate_kernel=GATE_TCGEN05):
    """Selected blocks idx [B, S, H, topk] int32 (ascending, -1 padded)."""
    _need(q, torch.bfloat16, "q")
    _need(kbar, torch.float32, "kbar")
    B, S, H, D = q.shape
    if block_size > 0 and tuple(kbar.shape) != (B * num_blocks(S, block_size), H, D):
        raise ValueError("kbar must be [B * ceil(S / block_size), H, D] (as kpool returns it)")
    idx = torch.empty(B, S, H, topk, dtype=torch.int32, device=q.device)
    o, _keep = _options(gate_kernel=gate_kernel)
    _check(lib().moba_gate_topk_ex(_ptr(q), _ptr(kbar), _ptr(idx), B, H, S, D, block_size, topk,
                                   ctypes.byref(o), _stream(stream)), "moba_gate_topk")
    return idx


def gate_topk_varlen(q, kbar, cu_seqlens, block_size: int, topk: int, stream=None,
                     gate_kernel=GATE_TCGEN05):
    _need(q, torch.bfloat16, "q")
    _need(kbar, torch.float32, "kbar")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    total, H, D = q.shape
    idx = torch.empty(total, H, topk, dtype=torch.int32, device=q.device)
    o, _keep = _options(gate_kernel=gate_kernel)
    _check(lib().moba_gate_topk_varlen_ex(_ptr(q), _ptr(kbar), _ptr(idx), _ptr(cu_seqlens),
                                          cu_seqlens.numel() - 1, total, H, D, block_size, topk,
                                          ctypes.byref(o), _stream(stream)),
           "moba_gate_topk_varlen")
    return idx


def workspace_size(B, H, S, D, block_size, topk) -> int:
    return int(lib().moba_attn_fwd_workspace_size(B, H, S, D, block_size, topk))


def varlen_workspace_size(num_seqs, total, max_seqlen, H, D, block_size, topk) -> int:
    return int(lib().moba_attn_fwd_varlen_workspace_size(num_seqs, total, max_seqlen, H, D,
                                                         block_size, topk))


def _idx_buffer(idx_out, rows_shape, topk, like):
    if idx_out is None:
        return None
    return _out(idx_out, (*rows_shape, topk), torch.int32, like, "idx_out")


def attn_fwd(q, k, v, block_size: int, topk: int, out=None, lse=None, workspace=None,
             stream=None, idx_out=None, phase_events=None, **options):
    """MoBA forward for q, k, v [B, S, H, D] bf16 -> (out [B, S, H, D] bf16, lse [B, H, S] fp32).

    With ``workspace`` (a uint8 CUDA tensor of at least :func:`workspace_size`
    bytes) the call allocates nothing; otherwise the library allocates its
    scratch stream-ordered.  ``idx_out`` ([B, S, H, topk] int32) receives the
    selection the call used; ``phase_events`` (see :func:`phase_events`) are
    recorded between its phases; further keyword ``options`` (pooling,
    gate_kernel, attn_kernel, debug_flags, wait_limit_cycles) are per call."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    B, S, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must have the same shape")
    out = _out(out, q.shape, torch.bfloat16, q, "out")
    lse = _out(lse, (B, H, S), torch.float32, q, "lse")
    workspace = _ws(workspace)
    idx_out = _idx_buffer(idx_out, (B, S, H), topk, q)
    o, _keep = _options(idx_out=idx_out, phase_events=phase_events, **options)
    rc = lib().moba_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                block_size, topk, ctypes.byref(o), _ptr(workspace),
                                workspace.numel() if workspace is not None else 0,
                                _stream(stream))
    _check(rc, "moba_attn_fwd")
    return out, lse


def host_scratch_size(B: int, H: int, S: int, D: int, block_size: int, topk: int) -> int:
    """Bytes of device scratch :func:`attn_fwd_host` needs."""
    return int(lib().moba_attn_fwd_host_scratch_size(B, H, S, D, block_size, topk))


def attn_fwd_host(q, k, v, block_size: int, topk: int, out, lse, scratch, stream=None,
                  **options):
    """The forward on host tensors (page-locked for asynchronous copies): q, k,
    v [B, S, H, D] bf16 in, out [B, S, H, D] bf16 and lse [B, H, S] fp32 filled
    in once ``stream`` has reached the end of the call's work.  ``scratch`` is a
    uint8 CUDA tensor of at least :func:`host_scratch_size` bytes; the library
    copies the inputs in and the results out itself."""
    for t, n, dt in ((q, "q", torch.bfloat16), (k, "k", torch.bfloat16),
                     (v, "v", torch.bfloat16), (out, "out", torch.bfloat16),
                     (lse, "lse", torch.float32)):
        if t.dtype != dt or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host {dt} tensor")
    B, S, H, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or out.shape != q.shape or \
            tuple(lse.shape) != (B, H, S):
        raise ValueError("q, k, v, out must be [B, S, H, D] and lse [B, H, S]")
    _need(scratch, torch.uint8, "scratch")
    o, _keep = _options(**options)
    rc = lib().moba_attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S, D,
                                  block_size, topk, ctypes.byref(o), _ptr(scratch),
                                  scratch.numel(), _stream(stream))
    _check(rc, "moba_attn_fwd_host")
    return out, lse


def decode_workspace_size(B: int, H: int, D: int, topk: int) -> int:
    return int(lib().moba_decode_workspace_size(B, H, D, topk))


def decode_fwd(q, k_cache, v_cache, kbar, cache_lens, block_size: int, topk: int, out=None,
               lse=None, idx=None, workspace=None, stream=None):
    """One decode step: q [B, H, D] bf16 against k_cache, v_cache [B, S_max, H,
    D] bf16 (the new token already at position cache_lens[b] - 1), kbar the
    caches' pooled keys (:func:`kpool` of k_cache), cache_lens int32 [B] on the
    device -> (out [B, H, D] bf16, lse [B, H] fp32, idx [B, H, topk] int32)."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(kbar, torch.float32, "kbar")
    _need(cache_lens, torch.int32, "cache_lens")
    B, H, D = q.shape
    if k_cache.dim() != 4 or k_cache.shape[0] != B or k_cache.shape[2:] != (H, D) or \
            v_cache.shape != k_cache.shape:
        raise ValueError("k_cache, v_cache must be [B, S_max, H, D] matching q")
    S_max = k_cache.shape[1]
    if block_size > 0 and tuple(kbar.shape) != (B * num_blocks(S_max, block_size), H, D):
        raise ValueError("kbar must be [B * ceil(S_max / block_size), H, D] (kpool of k_cache)")
    out = _out(out, q.shape, torch.bfloat16, q, "out")
    lse = _out(lse, (B, H), torch.float32, q, "lse")
    idx = _out(idx, (B, H, topk), torch.int32, q, "idx")
    workspace = _ws(workspace)
    st = _stream(stream)
    args = (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kbar), _ptr(cache_lens), _ptr(out),
            _ptr(lse), _ptr(idx), B, H, S_max, D, block_size, topk)
    if workspace is None:
        rc = lib().moba_decode_fwd(*args, st)
    else:
        rc = lib().moba_decode_fwd_ws(*args, _ptr(workspace), workspace.numel(), st)
    _check(rc, "moba_decode_fwd")
    return out, lse, idx


def attn_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, block_size: int, topk: int, out=None,
                    lse=None, workspace=None, stream=None, idx_out=None, phase_events=None,
                    **options):
    """Varlen MoBA forward: q, k, v [total, H, D] bf16, cu_seqlens int32 CUDA
    [num_seqs + 1] -> (out [total, H, D] bf16, lse [H, total] fp32).  Options
    as for :func:`attn_fwd` (``idx_out`` is [total, H, topk])."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    total, H, D = q.shape
    ns = cu_seqlens.numel() - 1
    for t, n in ((k, "k"), (v, "v")):
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    out = _out(out, q.shape, torch.bfloat16, q, "out")
    lse = _out(lse, (H, total), torch.float32, q, "lse")
    workspace = _ws(workspace)
    idx_out = _idx_buffer(idx_out, (total, H), topk, q)
    o, _keep = _options(idx_out=idx_out, phase_events=phase_events, **options)
    rc = lib().moba_attn_fwd_varlen_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                       _ptr(cu_seqlens), ns, total, max_seqlen, H, D,
                                       block_size, topk, ctypes.byref(o), _ptr(workspace),
                                       workspace.numel() if workspace is not None else 0,
                                       _stream(stream))
    _check(rc, "moba_attn_fwd_varlen")
    return out, lse


def bwd_workspace_size(B, H, S, D, block_size, topk) -> int:
    return int(lib().moba_attn_bwd_workspace_size(B, H, S, D, block_size, topk))


def attn_bwd(q, k, v, out, lse, dout, block_size: int, topk: int, dq=None, dk=None, dv=None,
             workspace=None, stream=None, **options):
    """MoBA backward for the forward ``attn_fwd(q, k, v, block_size, topk)``:
    q, k, v, out, dout [B, S, H, D] bf16 and lse [B, H, S] fp32 (as the forward
    returned them) -> (dq, dk, dv) [B, S, H, D] bf16.  The gate's selection is
    recomputed (with the same ``options`` as the forward) and held fixed, or,
    with ``idx_in`` ([B, S, H, topk] int32, the forward's ``idx_out``), taken
    as it is."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    _need(lse, torch.float32, "lse")
    B, S, H, D = q.shape
    for t, n in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    if tuple(lse.shape) != (B, H, S):
        raise ValueError("lse must be [B, H, S]")
    dq = _out(dq, q.shape, torch.bfloat16, q, "dq")
    dk = _out(dk, q.shape, torch.bfloat16, q, "dk")
    dv = _out(dv, q.shape, torch.bfloat16, q, "dv")
    workspace = _ws(workspace)
    o, _keep = _options(**options)
    rc = lib().moba_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, H, S, D, block_size, topk,
                                ctypes.byref(o), _ptr(workspace),
                                workspace.numel() if workspace is not None else 0,
                                _stream(stream))
    _check(rc, "moba_attn_bwd")
    return dq, dk, dv


def attn_bwd_varlen(q, k, v, out, lse, dout, cu_seqlens, max_seqlen: int, block_size: int,
                    topk: int, stream=None, **options):
    """Varlen backward: q, k, v, out, dout [total, H, D] bf16, lse [H, total]
    fp32, cu_seqlens int32 CUDA [num_seqs + 1] -> (dq, dk, dv) [total, H, D]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    _need(lse, torch.float32, "lse")
    _need(cu_seqlens, torch.int32, "cu_seqlens")
    total, H, D = q.shape
    ns = cu_seqlens.numel() - 1
    for t, n in ((k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    if tuple(lse.shape) != (H, total):
        raise ValueError("lse must be [H, total]")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    o, _keep = _options(**options)
    rc = lib().moba_attn_bwd_varlen_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                       _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens),
                                       ns, total, max_seqlen, H, D, block_size, topk,
                                       ctypes.byref(o), None, 0, _stream(stream))
    _check(rc, "moba_attn_bwd_varlen")
    return dq, dk, dv


def get_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib().moba_get_status(_stream(stream)))


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().moba_launch_count())


def attn_fwd_noalloc(q, k, v, block_size: int, topk: int, out, lse, stream=None):
    """moba_attn_fwd without any device allocation: the scratch is the
    library's static device array (see include/moba.h); `out` and `lse` must be
    provided by the caller."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _need(t, torch.bfloat16, n)
    _need(lse, torch.float32, "lse")
    B, S, H, D = q.shape
    for t, n in ((k, "k"), (v, "v"), (out, "out")):
        if t.shape != q.shape:
            raise ValueError(f"{n} must have the shape of q")
    if tuple(lse.shape) != (B, H, S):
        raise ValueError("lse must be [B, H, S]")
    _check(lib().moba_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, S,
                                       D, block_size, topk, _stream(stream)),
           "moba_attn_fwd_noalloc")
    return out, lse


def noalloc_capacity() -> int:
    return int(lib().moba_attn_fwd_noalloc_capacity())


def debug_timeout_info():
    """(barrier address, parity, block, thread) of the last reported timeout."""
    buf = (ctypes.c_int * 4)()
    lib().moba_debug_timeout_info(ctypes.cast(buf, ctypes.c_void_p))
    return tuple(buf)


# ---------------------------------------------------------------------------
# rotary positions and the paged cache
# ---------------------------------------------------------------------------
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BASE = 2
ROPE_BANDS = 3

@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


# the current stream's handle: torch's own short way where it has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _call(device: int, stream, fn):
    """fn(raw stream) with the tensors' device current, and ``stream`` too if one
    is given, so that results and scratch are allocated where they are used."""
    if stream is None and torch.cuda.current_device() == device:
        return fn(_raw_stream(device))
    if stream is not None and stream.device.index != device:
        raise ValueError(f"stream must be on cuda:{device}")
    with _switched(device, stream):
        return fn(torch.cuda.current_stream().cuda_stream)


# The checks of these calls are on a decode step's latency path: a tensor's
# device number says in one look that it is a CUDA tensor and on which device.
def _is(t, dtype, device) -> bool:
    return t.dtype is dtype and t.get_device() == device and t.is_contiguous()


def _tensor(t, dtype, device, name):
    if not _is(t, dtype, device):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor"
                         + (f" on cuda:{device}" if device >= 0 else ""))


def _device(t, name) -> int:
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return device


def _result(t, shape, dtype, like, device, name):
    """A result: a new tensor beside ``like``, or the caller's one, checked."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if not _is(t, dtype, device) or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on cuda:{device}")
    return t


def _heads(t, device, name):
    """(tokens, H, D, elements between tokens) of t [..., H, D] bf16: a token's
    heads dense, all tokens one stride apart."""
    if t.dtype is not torch.bfloat16 or t.get_device() != device or t.dim() < 2:
        raise ValueError(f"{name} must be a torch.bfloat16 tensor [..., H, D] on cuda:{device}")
    H, D = t.shape[-2:]
    if t.is_contiguous():
        return t.numel() // max(1, H * D), H, D, H * D
    stride, size, tokens = None, 1, 1
    if (D > 1 and t.stride(-1) != 1) or (H > 1 and t.stride(-2) != D):
        raise ValueError(f"{name}: a token's heads must be dense")
    for n, s in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
        tokens *= n
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != stride * size:
            raise ValueError(f"{name}: tokens must be one stride apart")
        size *= n
    if stride is not None and stride < H * D:
        raise ValueError(f"{name}: tokens must not overlap")
    return tokens, H, D, stride if stride is not None else H * D


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling=ROPE_PLAIN, factor: float = 1.0,
                     original_length: float = 0.0, slow_turns: float = 1.0,
                     fast_turns: float = 4.0, device="cuda"):
    """Radians per position of each pair of ``rot_dim`` rotated values: float64
    [rot_dim / 2] on ``device``; the scalings are those of moba_rope_frequencies
    (``ROPE_PLAIN``, ``ROPE_LINEAR``, ``ROPE_BASE``, ``ROPE_BANDS``)."""
    f = torch.empty(max(0, int(rot_dim)) // 2, dtype=torch.float64)
    _check(lib().moba_rope_frequencies(_ptr(f) if f.numel() else None, int(rot_dim), base, scaling,
                                       factor, original_length, slow_turns, fast_turns),
           "moba_rope_frequencies")
    return f.to(device)


def _rope(fn, what, q, k, positions, freqs, interleaved, magnitude, q_out, k_out, stream):
    device = _device(q, "q")
    T, Hq, D, qs = _heads(q, device, "q")
    _tensor(positions, torch.int32, device, "positions")
    _tensor(freqs, torch.float64, device, "freqs")
    if positions.numel() != T:
        raise ValueError(f"positions must hold one position for each of the {T} tokens")
    Hk = ks = 0
    if k is not None:
        Tk, Hk, Dk, ks = _heads(k, device, "k")
        if Tk != T or Dk != D:
            raise ValueError("k must have the tokens and the head dimension of q")
    elif k_out is not None:
        raise ValueError("k_out without k")

    def run(st):
        qo, ko, qos, kos, pk, pko = q_out, k_out, 0, 0, None, None
        if qo is None:
            qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif qo.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
        else:
            qos = _heads(qo, device, "q_out")[3]
        if k is not None:
            if ko is None:
                ko = torch.empty(k.shape, dtype=k.dtype, device=k.device)
            elif ko.shape != k.shape:
                raise ValueError("k_out must have the shape of k")
            else:
                kos = _heads(ko, device, "k_out")[3]
            pk, pko = k.data_ptr(), ko.data_ptr()
        if T == 0:
            return qo, ko
        rc = fn(q.data_ptr(), pk, qo.data_ptr(), pko, positions.data_ptr(), freqs.data_ptr(), T, Hq,
                Hk, D, 2 * freqs.numel(), 1 if interleaved else 0, magnitude, qs, ks, qos, kos, st)
        if rc:
            _check(rc, what)
        return qo, ko

    return _call(device, stream, run)


def rope(q, k, positions, freqs, interleaved: bool = False, magnitude: float = 1.0, q_out=None,
         k_out=None, stream=None):
    """Rotary positions: q [..., Hq, D] and k [..., Hk, D] bf16 (k may be None)
    with the first ``2 * len(freqs)`` values of each head rotated by
    ``positions[t] * freqs`` -> (q_out, k_out).  positions int32, one per token;
    freqs float64 (:func:`rope_frequencies`).  Pairs are (i, i + half), or
    (2i, 2i + 1) when ``interleaved``.  The tokens of an operand may be a stride
    apart (slices of one projection); q_out / k_out may be q / k (in place).
    No tokens: empty results, as of the other calls here."""
    return _rope(lib().moba_rope, "moba_rope", q, k, positions, freqs, interleaved, magnitude,
                 q_out, k_out, stream)


def rope_bwd(dq_out, dk_out, positions, freqs, interleaved: bool = False, magnitude: float = 1.0,
             dq=None, dk=None, stream=None):
    """The gradient of :func:`rope`: gradients of its outputs -> (dq, dk)."""
    return _rope(lib().moba_rope_bwd, "moba_rope_bwd", dq_out, dk_out, positions, freqs,
                 interleaved, magnitude, dq, dk, stream)


def _paged(device, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens):
    """Checks one layer's pools and the sequences' tables; the sizes a call passes on."""
    bf16, i32 = torch.bfloat16, torch.int32
    _tensor(k_pages, bf16, device, "k_pages")
    _tensor(v_pages, bf16, device, "v_pages")
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, D]")
    P, Hkv, ps, D = shape
    bar = None
    if kbar_pages is not None:
        _tensor(kbar_pages, torch.float32, device, "kbar_pages")
        if kbar_pages.shape != (P, Hkv, D):
            raise ValueError("kbar_pages must be [num_pages, Hkv, D]")
        bar = kbar_pages.data_ptr()
    _tensor(page_table, i32, device, "page_table")
    _tensor(cu_new, i32, device, "cu_new")
    _tensor(cache_lens, i32, device, "cache_lens")
    n = cache_lens.numel()
    table = page_table.shape
    if len(table) != 2 or table[0] != n or cu_new.numel() != n + 1:
        raise ValueError("page_table must be [num_seqs, max_pages], cu_new [num_seqs + 1] and "
                         "cache_lens [num_seqs]")
    return P, Hkv, ps, D, n, table[1], bar


def paged_append(k, v, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens, max_new: int,
                 block_size: int, pooling=POOL_MEAN, stream=None):
    """Writes the new tokens' k, v [total, Hkv, D] bf16 to the pages of their
    sequences (the last ``cu_new[b + 1] - cu_new[b]`` of ``cache_lens[b]`` tokens) and
    the pooled keys of the blocks that they complete to ``kbar_pages`` (None: the
    cache keeps none)."""
    device = _device(k_pages, "k_pages")
    P, Hkv, ps, D, n, mp, bar = _paged(device, k_pages, v_pages, kbar_pages, page_table, cu_new,
                                       cache_lens)
    _tensor(k, torch.bfloat16, device, "k")
    _tensor(v, torch.bfloat16, device, "v")
    shape = k.shape
    if len(shape) != 3 or shape[1] != Hkv or shape[2] != D or v.shape != shape:
        raise ValueError("k and v must be [total, Hkv, D] of the pages")
    if shape[0] == 0:
        return
    opt = ctypes.byref(_options(pooling=pooling)[0]) if pooling != POOL_MEAN else None
    rc = _call(device, stream, lambda st: lib().moba_paged_append(
        k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), bar,
        page_table.data_ptr(), cu_new.data_ptr(), cache_lens.data_ptr(), n, shape[0], max_new, Hkv,
        D, P, ps, mp, block_size, opt, st))
    if rc:
        _check(rc, "moba_paged_append")


def paged_attn_workspace_size(num_seqs, total, max_new, Hq, Hkv, D, page_size, max_pages,
                              block_size, topk) -> int:
    """Bytes of scratch :func:`paged_attn` needs on the current device (0: sizes it refuses)."""
    return int(lib().moba_paged_attn_workspace_size(num_seqs, total, max_new, Hq, Hkv, D, page_size,
                                                    max_pages, block_size, topk))


def paged_attn(q, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens, max_new: int,
               block_size: int, topk: int, out=None, lse=None, idx=None, with_idx: bool = False,
               workspace=None, stream=None):
    """Attention of the new tokens q [total, Hq, D] bf16 (already appended, see
    :func:`paged_append`) over the paged cache -> (out [total, Hq, D] bf16, lse
    [total, Hq] fp32, idx [total, Hq, topk] int32 or None): MoBA over the own
    block and the best topk - 1 past blocks of each query head, or full causal
    attention when topk covers the blocks of a page table row.  ``workspace`` is
    a uint8 CUDA tensor of at least :func:`paged_attn_workspace_size` bytes, or
    None (scratch from torch's allocator, on the call's stream)."""
    device = _device(k_pages, "k_pages")
    P, Hkv, ps, D, n, mp, bar = _paged(device, k_pages, v_pages, kbar_pages, page_table, cu_new,
                                       cache_lens)
    _tensor(q, torch.bfloat16, device, "q")
    shape = q.shape
    if len(shape) != 3 or shape[2] != D:
        raise ValueError("q must be [total, Hq, D] with the pages' head dimension")
    total, Hq = shape[0], shape[1]
    if workspace is not None:
        _tensor(workspace, torch.uint8, device, "workspace")

    def run(st):
        ws = workspace
        if ws is None:
            size = lib().moba_paged_attn_workspace_size(n, total, max_new, Hq, Hkv, D, ps, mp,
                                                        block_size, topk)
            ws = torch.empty(size, dtype=torch.uint8, device=q.device)
        o = _result(out, shape, torch.bfloat16, q, device, "out")
        z = _result(lse, (total, Hq), torch.float32, q, device, "lse")
        sel = None
        if with_idx or idx is not None:
            sel = _result(idx, (total, Hq, topk), torch.int32, q, device, "idx")
        if total == 0:
            return o, z, sel
        rc = lib().moba_paged_attn(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), bar, page_table.data_ptr(),
            cu_new.data_ptr(), cache_lens.data_ptr(), o.data_ptr(), z.data_ptr(),
            sel.data_ptr() if sel is not None else None, n, total, max_new, Hq, Hkv, D, P, ps, mp,
            block_size, topk, ws.data_ptr(), ws.numel(), st)
        if rc:
            _check(rc, "moba_paged_attn")
        return o, z, sel

    return _call(device, stream, run)


def page_copy(k_pages, v_pages, kbar_pages, src, dst, stream=None):
    """Copies pages ``src[i]`` to ``dst[i]`` (int32) of the pools [num_pages, Hkv,
    page_size, D] (kbar_pages [num_pages, Hkv, D] or None), or of every layer of
    pools with a leading layer dimension."""
    device = _device(k_pages, "k_pages")
    _tensor(k_pages, torch.bfloat16, device, "k_pages")
    _tensor(v_pages, torch.bfloat16, device, "v_pages")
    shape = k_pages.shape
    if len(shape) not in (4, 5) or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must be [(layers,) num_pages, Hkv, page_size, D]")
    P, Hkv, ps, D = shape[-4:]
    bar = None
    if kbar_pages is not None:
        _tensor(kbar_pages, torch.float32, device, "kbar_pages")
        if kbar_pages.shape != (*shape[:-2], D):
            raise ValueError("kbar_pages must be [(layers,) num_pages, Hkv, D]")
        bar = kbar_pages.data_ptr()
    _tensor(src, torch.int32, device, "src")
    _tensor(dst, torch.int32, device, "dst")
    n = src.numel()
    if n != dst.numel():
        raise ValueError("src and dst must have the same length")
    if n == 0:
        return
    layers = shape[0] if len(shape) == 5 else 1
    rc = _call(device, stream, lambda st: lib().moba_page_copy(
        k_pages.data_ptr(), v_pages.data_ptr(), bar, src.data_ptr(), dst.data_ptr(), n, layers, P,
        Hkv, D, ps, st))
    if rc:
        _check(rc, "moba_page_copy")
