"""Thin ctypes binding of libattnres.so (C ABI in include/attnres.h).

Argument marshalling only: every step of the read runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (torch supplies device memory and the
current stream); each function has the name of the C entry point it calls and
raises ``AttnResError`` when the call does not return ATTNRES_OK.  There is no
fallback: if the library is missing, the first call raises.

``stream``: the stream of the call's kernels instead of the current one, as if the
call were made under ``torch.cuda.stream(stream)``: outputs and workspaces that it
allocates belong to that stream too.  The caller orders it with the streams that
write the inputs and use the outputs.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import functools
import inspect
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libattnres.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "attnres.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT = range(5)
F32, BF16 = 0, 1
CACHE_FP4, CACHE_FP8 = 0, 1     # formats of the quantised depth cache

_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_f = ctypes.c_float
_SIGS = {
    "attnres_full_fwd": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _f, _vp, _vp],
    "attnres_block_phase1": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, _vp,
                             _vp, _vp],
    "attnres_block_phase2_merge": [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp, _f, _vp, _vp],
    "attnres_block_phase2_update_merge": [_vp, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp,
                                          _f, _vp, _vp],
    "mhar_phase2_merge": [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _f, _vp, _vp],
    "attnres_read_bwd": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, _vp, _vp, _i64,
                         ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "attnres_read_bwd_noalloc": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, _vp, _vp, _i64,
                                 ctypes.c_int, _vp, _vp, _vp],
    "attnres_read_bwd_workspace_size": [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "attnres_block_phase1_bwd": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, _vp, _vp, _vp,
                                 _i64, ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "attnres_block_phase2_bwd": [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _vp, _f, _vp, _vp, _vp, _vp,
                                 ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "attnres_block_phase2_bwd_workspace_size": [_i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "mhar_read_bwd": [_vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, _vp, _vp, _i64,
                      ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "mhar_read_bwd_workspace_size": [_i64, _i64, _i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "mhar_fwd": [_vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, _vp, _vp,
                 _vp],
    "msar_expand_fwd": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f,
                        _vp, _vp, _f, _vp, _vp],
    "msar_expand_fwd_ps": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _i64, _vp, _vp, _f, _vp,
                           _vp, _f, _vp, _vp],
    "msar_block_phase1": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _i64, _vp, _f, _vp,
                          _vp, _vp],
    "msar_block_phase2": [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f, _vp, _vp, _f,
                          _vp, _vp],
    "msar_expand_fwd_chunk": [_vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f,
                              _vp, _vp, _f, _vp, _vp],
    "msar_expand_bwd": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f, _vp, _vp, _f,
                        _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "msar_expand_bwd_workspace_size": [_i64, _i64, _i64, ctypes.c_int, _i64, _vp, ctypes.POINTER(ctypes.c_size_t)],
    "msar_expand_bwd_chunk": [_vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f, _vp,
                              _vp, _f, _vp, _vp, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                              _vp],
    "msar_expand_bwd_ps": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _i64, _vp, _vp, _f, _vp, _vp,
                           _f, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "msar_expand_fwd_ws": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _i64, _vp, _vp, _f, _vp, _vp,
                           _f, _vp, _vp, ctypes.c_size_t, _vp],
    "msar_expand_fwd_ws_workspace_size": [_i64, _i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "msar_block_phase1_ws": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _i64, _vp, _f, _vp,
                             _vp, _vp, ctypes.c_size_t, _vp],
    "msar_block_phase1_ws_workspace_size": [_i64, _i64, _i64, ctypes.c_int, _i64, ctypes.POINTER(ctypes.c_size_t)],
    "msar_block_phase2_ws": [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f, _vp, _vp, _f,
                             _vp, _vp, ctypes.c_size_t, _vp],
    "msar_block_phase2_ws_workspace_size": [_i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "msar_block_phase2_bwd": [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _f, _vp, _vp, _f,
                              _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "msar_block_phase2_bwd_workspace_size": [_i64, _i64, ctypes.c_int, _i64, _vp, ctypes.POINTER(ctypes.c_size_t)],
    "msar_block_phase1_bwd": [_vp, _i64, _i64, _i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _i64, _vp, _f, _vp,
                              _vp, _vp, _i64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "msar_block_phase1_bwd_workspace_size": [_i64, _i64, _i64, ctypes.c_int, _i64, _vp, _i64,
                                             ctypes.POINTER(ctypes.c_size_t)],
    "attnres_cache_row_bytes": [ctypes.c_int, _i64, _i64, ctypes.POINTER(ctypes.c_size_t)],
    "attnres_cache_quant": [_vp, _vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, _i64, _vp],
    "attnres_cache_dequant": [_vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp, _i64, _vp],
    "attnres_cache_read": [_vp, _i64, _i64, _i64, _i64, _i64, ctypes.c_int, _vp, _i64, _vp, _f, ctypes.c_int, _vp,
                           _vp, _vp],
    "attnres_phase2_norm_q8": [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_int, _vp, _vp, _f, _vp, _f, _i64,
                               _vp, _vp, _vp, _vp],
    "attnres_norm_bwd": [_vp, _vp, _vp, _i64, _i64, ctypes.c_int, _vp, _f, _vp, _vp, _vp, ctypes.c_size_t, _vp],
    "attnres_norm_bwd_workspace_size": [_i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)],
    "attnres_status_string": [ctypes.c_int],
    "attnres_last_cuda_error": [],
    "attnres_sync_status": [_vp],
    "attnres_debug_set_wait_timeout_ns": [ctypes.c_uint64],
    "attnres_debug_set_stall_injection": [ctypes.c_int],
    "attnres_debug_set_kernel_variant": [ctypes.c_int],
    "attnres_version": [],
}
_RESTYPES = {"attnres_status_string": ctypes.c_char_p, "attnres_last_cuda_error": ctypes.c_char_p,
             "attnres_version": ctypes.c_char_p, "attnres_debug_set_wait_timeout_ns": None,
             "attnres_debug_set_stall_injection": None,
             "attnres_debug_set_kernel_variant": None}


class AttnResError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn}: {status_string(status)}"
        if status == ERR_CUDA:
            msg += f" ({last_cuda_error()})"
        super().__init__(msg)


def load(path: str = LIB_PATH):
    """Load libattnres.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m depth_wise_attention_gb300.build`")
        lib = ctypes.CDLL(path)
        for name, args in _SIGS.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = _RESTYPES.get(name, ctypes.c_int)
        _lib = lib
    return _lib


def header_functions(header: str = HEADER):
    """Names of the functions declared in include/attnres.h."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b([a-z_0-9]+)\s*\(", text)) - {"defined"})


def status_string(status: int) -> str:
    return load().attnres_status_string(status).decode()


def last_cuda_error() -> str:
    return load().attnres_last_cuda_error().decode()


def version() -> str:
    return load().attnres_version().decode()


def _dt(t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    return None if t is None else _vp(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return _vp(s.cuda_stream)


def _on_stream(fn):
    """Runs fn under the `stream` that it is given.  Memory of the caching allocator goes by the stream that is
    current when it is allocated: what fn allocates on another stream than that of its kernels could still be in
    use there, and would be handed out again there while the kernels use it."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        import torch
        dev = stream.device_index
        if dev != torch._C._cuda_getDevice():
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        # what that context does on the current device, at a tenth of its 10 us
        before = torch._C._cuda_getCurrentStream(dev)
        if before[0] == stream.stream_id:
            return fn(*args, **kw)
        torch._C._cuda_setStream(stream_id=stream.stream_id, device_index=dev, device_type=stream.device_type)
        try:
            return fn(*args, **kw)
        finally:
            torch._C._cuda_setStream(stream_id=before[0], device_index=before[1], device_type=before[2])
    return call


def _check(fn, status):
    if status != OK:
        raise AttnResError(fn, status)


def _src_geometry(src):
    """src [n_src, T, d]: each source contiguous, sources src.stride(0) apart."""
    n_src, T, d = src.shape
    if src.stride(2) != 1 or src.stride(1) != d:
        raise ValueError("each source must be a contiguous [T, d] block")
    return n_src, T, d, src.stride(0)


@_on_stream
def attnres_full_fwd(src, query, gain=None, eps=1e-6, out=None, stream=None):
    """Full AttnRes read of one layer: src [n_src,T,d] -> out [T,d]."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    if out is None:
        out = torch.empty((T, d), dtype=src.dtype, device=src.device)
    _check("attnres_full_fwd", load().attnres_full_fwd(
        _p(src), n_src, stride, T, d, _dt(src), _p(query), _p(gain), eps, _p(out), _stream(stream)))
    return out


@_on_stream
def attnres_block_phase1(src, queries, gain=None, eps=1e-6, o=None, lse=None, want_lse=True,
                         stream=None):
    """Phase 1: queries [n_q,d] against src [n_src,T,d] -> (o [n_q,T,d], lse [n_q,T])."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    n_q = queries.shape[0]
    if o is None:
        o = torch.empty((n_q, T, d), dtype=src.dtype, device=src.device)
    if lse is None and want_lse:
        lse = torch.empty((n_q, T), dtype=torch.float32, device=src.device)
    _check("attnres_block_phase1", load().attnres_block_phase1(
        _p(src), n_src, stride, T, d, _dt(src), _p(queries), n_q, _p(gain), eps, _p(o), _p(lse),
        _stream(stream)))
    return o, lse


@_on_stream
def attnres_block_phase2_merge(o, lse, partial, query, gain=None, eps=1e-6, out=None, stream=None):
    """Phase 2: merge partial [T,d] (or None) into (o [T,d], lse [T]) -> out [T,d]."""
    import torch
    T, d = o.shape
    if out is None:
        out = torch.empty_like(o)
    _check("attnres_block_phase2_merge", load().attnres_block_phase2_merge(
        _p(o), _p(lse), _p(partial), T, d, _dt(o), _p(query), _p(gain), eps, _p(out),
        _stream(stream)))
    return out


@_on_stream
def attnres_block_phase2_update_merge(partial, f, o, lse, query, gain=None, eps=1e-6, partial_out=None,
                                      out=None, stream=None):
    """Fused update and merge: partial [T,d] or None, f [T,d] -> (partial + f, merged out).
    partial_out may be partial or f (in place); out may be o."""
    import torch
    T, d = o.shape
    if partial_out is None:
        partial_out = torch.empty_like(f)
    if out is None:
        out = torch.empty_like(o)
    _check("attnres_block_phase2_update_merge", load().attnres_block_phase2_update_merge(
        _p(partial), _p(f), _p(partial_out), _p(o), _p(lse), T, d, _dt(o), _p(query), _p(gain), eps,
        _p(out), _stream(stream)))
    return partial_out, out


@_on_stream
def mhar_phase2_merge(o, lse, partial, query, gain=None, eps=1e-6, f=None, partial_out=None, out=None,
                      stream=None):
    """Per-head phase-2 merge: o [T,d], lse [H,T], partial [T,d] or None, query [H,d/H].
    With f, the partial is first updated (returned as partial_out).  Returns out, or
    (partial_out, out) when f is given."""
    import torch
    T, d = o.shape
    H = query.shape[0]
    if f is not None and partial_out is None:
        partial_out = torch.empty_like(f)
    if out is None:
        out = torch.empty_like(o)
    _check("mhar_phase2_merge", load().mhar_phase2_merge(
        _p(o), _p(lse), _p(partial), _p(f), _p(partial_out), T, d, H, _dt(o), _p(query), _p(gain), eps,
        _p(out), _stream(stream)))
    return (partial_out, out) if f is not None else out


def attnres_read_bwd_workspace_size(n_src, T, d, n_q, dtype):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    _check("attnres_read_bwd_workspace_size",
           load().attnres_read_bwd_workspace_size(n_src, T, d, n_q, dt, ctypes.byref(n)))
    return n.value


@_on_stream
def attnres_read_bwd(src, queries, dout, gain=None, eps=1e-6, dsrc=None, accumulate=False, dqueries=None,
                     dgain=None, want_dgain=True, workspace=None, stream=None):
    """Backward of the read of queries [n_q,d] over src [n_src,T,d] for output
    gradients dout [n_q,T,d] -> (dsrc, dqueries, dgain).  The workspace is
    allocated here unless given (the library itself allocates nothing)."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    n_q = queries.shape[0]
    if dsrc is None:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=src.device)
    _, _, _, dstride = _src_geometry(dsrc)
    if dqueries is None:
        dqueries = torch.empty((n_q, d), dtype=torch.float32, device=src.device)
    if dgain is None and want_dgain:
        dgain = torch.empty((d,), dtype=torch.float32, device=src.device)
    if workspace is None:
        nbytes = attnres_read_bwd_workspace_size(n_src, T, d, n_q, src.dtype)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=src.device)
    _check("attnres_read_bwd", load().attnres_read_bwd(
        _p(src), n_src, stride, T, d, _dt(src), _p(queries), n_q, _p(gain), eps, _p(dout), _p(dsrc), dstride,
        1 if accumulate else 0, _p(dqueries), _p(dgain), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return dsrc, dqueries, dgain


@_on_stream
def attnres_read_bwd_noalloc(src, queries, dout, gain=None, eps=1e-6, dsrc=None, accumulate=False,
                             dqueries=None, dgain=None, want_dgain=True, stream=None):
    """attnres_read_bwd with the library's built-in scratch instead of a workspace."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    n_q = queries.shape[0]
    if dsrc is None:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=src.device)
    _, _, _, dstride = _src_geometry(dsrc)
    if dqueries is None:
        dqueries = torch.empty((n_q, d), dtype=torch.float32, device=src.device)
    if dgain is None and want_dgain:
        dgain = torch.empty((d,), dtype=torch.float32, device=src.device)
    _check("attnres_read_bwd_noalloc", load().attnres_read_bwd_noalloc(
        _p(src), n_src, stride, T, d, _dt(src), _p(queries), n_q, _p(gain), eps, _p(dout), _p(dsrc), dstride,
        1 if accumulate else 0, _p(dqueries), _p(dgain), _stream(stream)))
    return dsrc, dqueries, dgain


@_on_stream
def attnres_block_phase1_bwd(src, queries, d_o, d_lse=None, gain=None, eps=1e-6, dsrc=None, accumulate=False,
                             dqueries=None, dgain=None, want_dgain=True, workspace=None, stream=None):
    """Backward of Block phase 1 for gradients of its outputs o [n_q,T,d] and
    lse [n_q,T] (None: zero) -> (dsrc, dqueries, dgain)."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    n_q = queries.shape[0]
    if dsrc is None:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=src.device)
    _, _, _, dstride = _src_geometry(dsrc)
    if dqueries is None:
        dqueries = torch.empty((n_q, d), dtype=torch.float32, device=src.device)
    if dgain is None and want_dgain:
        dgain = torch.empty((d,), dtype=torch.float32, device=src.device)
    if workspace is None:
        nbytes = attnres_read_bwd_workspace_size(n_src, T, d, n_q, src.dtype)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=src.device)
    _check("attnres_block_phase1_bwd", load().attnres_block_phase1_bwd(
        _p(src), n_src, stride, T, d, _dt(src), _p(queries), n_q, _p(gain), eps, _p(d_o), _p(d_lse), _p(dsrc),
        dstride, 1 if accumulate else 0, _p(dqueries), _p(dgain), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return dsrc, dqueries, dgain


def attnres_block_phase2_bwd_workspace_size(T, d, dtype):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    _check("attnres_block_phase2_bwd_workspace_size",
           load().attnres_block_phase2_bwd_workspace_size(T, d, dt, ctypes.byref(n)))
    return n.value


@_on_stream
def attnres_block_phase2_bwd(o, lse, partial, query, dh, gain=None, eps=1e-6, d_o=None, d_lse=None,
                             d_partial=None, accumulate=False, dquery=None, dgain=None, want_dgain=True,
                             workspace=None, stream=None):
    """Backward of the phase-2 merge: o, partial (or None), dh [T,d]; lse [T]
    -> (d_o, d_lse, d_partial (None without a partial), dquery, dgain)."""
    import torch
    T, d = o.shape
    if d_o is None:
        d_o = torch.empty_like(o)
    if d_lse is None:
        d_lse = torch.empty((T,), dtype=torch.float32, device=o.device)
    if partial is not None and d_partial is None:
        d_partial = torch.empty_like(partial)
    if dquery is None:
        dquery = torch.empty((d,), dtype=torch.float32, device=o.device)
    if dgain is None and want_dgain:
        dgain = torch.empty((d,), dtype=torch.float32, device=o.device)
    if workspace is None:
        nbytes = attnres_block_phase2_bwd_workspace_size(T, d, o.dtype)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=o.device)
    _check("attnres_block_phase2_bwd", load().attnres_block_phase2_bwd(
        _p(o), _p(lse), _p(partial), T, d, _dt(o), _p(query), _p(gain), eps, _p(dh), _p(d_o), _p(d_lse),
        _p(d_partial), 1 if accumulate else 0, _p(dquery), _p(dgain), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return d_o, d_lse, (d_partial if partial is not None else None), dquery, dgain


def mhar_read_bwd_workspace_size(n_src, T, d, H, n_q, dtype):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    _check("mhar_read_bwd_workspace_size",
           load().mhar_read_bwd_workspace_size(n_src, T, d, H, n_q, dt, ctypes.byref(n)))
    return n.value


@_on_stream
def mhar_read_bwd(src, queries, dout, gain=None, eps=1e-6, dsrc=None, accumulate=False, dqueries=None,
                  dgain=None, want_dgain=True, workspace=None, stream=None):
    """Backward of the MHAR read of queries [n_q,H,d/H] over src [n_src,T,d]
    for output gradients dout [n_q,T,d] -> (dsrc, dqueries [n_q,H,d/H],
    dgain).  The workspace is allocated here unless given."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    n_q, H, dh = queries.shape
    if H * dh != d:
        raise ValueError("queries must be [n_q, H, d/H]")
    if dsrc is None:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=src.device)
    _, _, _, dstride = _src_geometry(dsrc)
    if dqueries is None:
        dqueries = torch.empty((n_q, H, dh), dtype=torch.float32, device=src.device)
    if dgain is None and want_dgain:
        dgain = torch.empty((d,), dtype=torch.float32, device=src.device)
    if workspace is None:
        nbytes = mhar_read_bwd_workspace_size(n_src, T, d, H, n_q, src.dtype)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=src.device)
    _check("mhar_read_bwd", load().mhar_read_bwd(
        _p(src), n_src, stride, T, d, H, _dt(src), _p(queries), n_q, _p(gain), eps, _p(dout), _p(dsrc), dstride,
        1 if accumulate else 0, _p(dqueries), _p(dgain), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return dsrc, dqueries, dgain


@_on_stream
def mhar_fwd(src, queries, gain=None, eps=1e-6, out=None, lse=None, want_lse=False, stream=None):
    """MHAR: queries [n_q,H,d/H] -> out [n_q,T,d] (lse [n_q,H,T])."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    n_q, H, _ = queries.shape
    if out is None:
        out = torch.empty((n_q, T, d), dtype=src.dtype, device=src.device)
    if lse is None and want_lse:
        lse = torch.empty((n_q, H, T), dtype=torch.float32, device=src.device)
    _check("mhar_fwd", load().mhar_fwd(
        _p(src), n_src, stride, T, d, H, _dt(src), _p(queries), n_q, _p(gain), eps, _p(out), _p(lse),
        _stream(stream)))
    return (out, lse) if want_lse else out


@_on_stream
def msar_expand_fwd(src, ksizes, conv_w, queries, gain=None, eps=1e-6, mix_gain=None, mix_w=None,
                    mix_eps=1e-6, out=None, stream=None):
    """MSAR: src [n_src,T,d], ksizes (m-1 ints, host), conv_w packed, queries [m,d],
    mix_w [m*d,m] -> out [T,d]."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if out is None:
        out = torch.empty((T, d), dtype=src.dtype, device=src.device)
    _check("msar_expand_fwd", load().msar_expand_fwd(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries),
        _p(gain), eps, _p(mix_gain), _p(mix_w), mix_eps, _p(out), _stream(stream)))
    return out


def attnres_sync_status(stream=None):
    """Wait for the stream and raise if a kernel recorded a device-side timeout."""
    _check("attnres_sync_status", load().attnres_sync_status(_stream(stream)))


def attnres_debug_set_wait_timeout_ns(ns: int):
    load().attnres_debug_set_wait_timeout_ns(int(ns))


def attnres_debug_set_stall_injection(enable: int):
    load().attnres_debug_set_stall_injection(int(enable))


def attnres_debug_set_kernel_variant(variant: int):
    """0: automatic kernel choice; 1: always the general CUDA-core depth read;
    2: the tensor-core depth reads wherever they apply; 3: the few-token kernel
    (a token per cluster of CTAs) wherever it applies."""
    load().attnres_debug_set_kernel_variant(int(variant))


@_on_stream
def msar_expand_fwd_chunk(src, t_prev, ksizes, conv_w, queries, gain=None, eps=1e-6, mix_gain=None, mix_w=None,
                          mix_eps=1e-6, out=None, stream=None):
    """MSAR for one chunk: src [n_src, t_prev + T, d] (t_prev history rows first)
    -> out [T, d] for the last T rows."""
    import torch
    n_src, rows, d, stride = _src_geometry(src)
    T = rows - t_prev
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if out is None:
        out = torch.empty((T, d), dtype=src.dtype, device=src.device)
    _check("msar_expand_fwd_chunk", load().msar_expand_fwd_chunk(
        _p(src), n_src, stride, t_prev, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries),
        _p(gain), eps, _p(mix_gain), _p(mix_w), mix_eps, _p(out), _stream(stream)))
    return out


@_on_stream
def msar_block_phase1(src, ksizes, conv_w, queries, gain=None, eps=1e-6, o=None, lse=None, stream=None):
    """MSAR two-phase, phase 1: queries [S, m, d] of a block's layers over the
    cached sources src [n_src, T, d] -> (o [S, m, T, d], lse [S, m, T])."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    S, m, _ = queries.shape
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if o is None:
        o = torch.empty((S, m, T, d), dtype=src.dtype, device=src.device)
    if lse is None:
        lse = torch.empty((S, m, T), dtype=torch.float32, device=src.device)
    _check("msar_block_phase1", load().msar_block_phase1(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries), S, _p(gain),
        eps, _p(o), _p(lse), _stream(stream)))
    return o, lse


@_on_stream
def msar_block_phase2(o, lse, partial, ksizes, conv_w, query, gain=None, eps=1e-6, mix_gain=None, mix_w=None,
                      mix_eps=1e-6, out=None, stream=None):
    """MSAR two-phase, phase 2 of one layer: o [m, T, d], lse [m, T], partial
    [T, d] or None, query [m, d] -> out [T, d]."""
    import torch
    m, T, d = o.shape
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if out is None:
        out = torch.empty((T, d), dtype=o.dtype, device=o.device)
    _check("msar_block_phase2", load().msar_block_phase2(
        _p(o), _p(lse), _p(partial), T, d, _dt(o), m, ctypes.cast(ks, _vp), _p(conv_w), _p(query), _p(gain), eps,
        _p(mix_gain), _p(mix_w), mix_eps, _p(out), _stream(stream)))
    return out


@_on_stream
def msar_expand_fwd_ps(src, ksizes, conv_w, queries, gain=None, eps=1e-6, mix_gain=None, mix_w=None, mix_eps=1e-6,
                       out=None, stream=None):
    """MSAR with each source's own conv kernels: conv_w [n_src, d*sum(k)] (or
    any [n_src, stride >= d*sum(k)] float tensor) -> out [T, d]."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if out is None:
        out = torch.empty((T, d), dtype=src.dtype, device=src.device)
    _check("msar_expand_fwd_ps", load().msar_expand_fwd_ps(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), conv_w.stride(0), _p(queries),
        _p(gain), eps, _p(mix_gain), _p(mix_w), mix_eps, _p(out), _stream(stream)))
    return out


def msar_expand_bwd_workspace_size(n_src, T, d, dtype, ksizes):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    _check("msar_expand_bwd_workspace_size", load().msar_expand_bwd_workspace_size(
        n_src, T, d, dt, len(ksizes) + 1, ctypes.cast(ks, _vp), ctypes.byref(n)))
    return n.value


@_on_stream
def msar_expand_bwd(src, ksizes, conv_w, queries, dh, gain=None, eps=1e-6, mix_gain=None, mix_w=None, mix_eps=1e-6,
                    dsrc=None, want_dgain=True, want_dmix_gain=True, grads=None, workspace=None, stream=None):
    """Backward of msar_expand_fwd for dh [T,d] -> (dsrc [n_src,T,d], dconv_w
    (packed as conv_w), dqueries [m,d], dgain [d], dmix_gain [m*d], dmix_w
    [m*d,m]).  grads: the five parameter-gradient tensors to write (else
    allocated here, as is the workspace unless given)."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    dev = src.device
    if dsrc is None:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=dev)
    _, _, _, dstride = _src_geometry(dsrc)
    if grads is not None:
        dconv_w, dqueries, dgain, dmix_gain, dmix_w = grads
    else:
        dconv_w = torch.empty_like(conv_w, dtype=torch.float32)
        dqueries = torch.empty((m, d), dtype=torch.float32, device=dev)
        dgain = torch.empty((d,), dtype=torch.float32, device=dev) if want_dgain else None
        dmix_gain = torch.empty((m * d,), dtype=torch.float32, device=dev) if want_dmix_gain else None
        dmix_w = torch.empty((m * d, m), dtype=torch.float32, device=dev)
    if workspace is None:
        nbytes = msar_expand_bwd_workspace_size(n_src, T, d, src.dtype, ksizes)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=dev)
    _check("msar_expand_bwd", load().msar_expand_bwd(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries), _p(gain), eps,
        _p(mix_gain), _p(mix_w), mix_eps, _p(dh), _p(dsrc), dstride, _p(dconv_w), _p(dqueries), _p(dgain),
        _p(dmix_gain), _p(dmix_w), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return dsrc, dconv_w, dqueries, dgain, dmix_gain, dmix_w


@_on_stream
def msar_expand_bwd_ps(src, ksizes, conv_w, queries, dh, gain=None, eps=1e-6, mix_gain=None, mix_w=None,
                       mix_eps=1e-6, dsrc=None, want_dgain=True, want_dmix_gain=True, grads=None, workspace=None,
                       stream=None):
    """Backward of msar_expand_fwd_ps: conv_w [n_src, stride >= d*sum(k)] ->
    (dsrc, dconv_w [n_src, stride] (each source's own; the padding past
    d*sum(k) is zero), dqueries, dgain, dmix_gain, dmix_w)."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    dev = src.device
    if dsrc is None:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=dev)
    _, _, _, dstride = _src_geometry(dsrc)
    if grads is not None:
        dconv_w, dqueries, dgain, dmix_gain, dmix_w = grads
    else:
        dconv_w = torch.zeros(conv_w.shape, dtype=torch.float32, device=dev)
        dqueries = torch.empty((m, d), dtype=torch.float32, device=dev)
        dgain = torch.empty((d,), dtype=torch.float32, device=dev) if want_dgain else None
        dmix_gain = torch.empty((m * d,), dtype=torch.float32, device=dev) if want_dmix_gain else None
        dmix_w = torch.empty((m * d, m), dtype=torch.float32, device=dev)
    if workspace is None:
        nbytes = msar_expand_bwd_workspace_size(n_src, T, d, src.dtype, ksizes)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=dev)
    _check("msar_expand_bwd_ps", load().msar_expand_bwd_ps(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), conv_w.stride(0), _p(queries),
        _p(gain), eps, _p(mix_gain), _p(mix_w), mix_eps, _p(dh), _p(dsrc), dstride, _p(dconv_w), _p(dqueries),
        _p(dgain), _p(dmix_gain), _p(dmix_w), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return dsrc, dconv_w, dqueries, dgain, dmix_gain, dmix_w


def msar_expand_fwd_ws_workspace_size(n_src, T, d, dtype):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    _check("msar_expand_fwd_ws_workspace_size",
           load().msar_expand_fwd_ws_workspace_size(n_src, T, d, dt, ctypes.byref(n)))
    return n.value


@_on_stream
def msar_expand_bwd_chunk(src, t_prev, ksizes, conv_w, queries, dh, dsrc, grads, accumulate, gain=None, eps=1e-6,
                          mix_gain=None, mix_w=None, mix_eps=1e-6, workspace=None, stream=None):
    """Backward of one chunk: src [n_src, t_prev + T, d] (t_prev history rows
    first), dh [T, d]; dsrc [n_src, t_prev + T, d] gets the chunk's rows
    written and the history rows' share added; grads = (dconv_w, dqueries,
    dgain, dmix_gain, dmix_w) are written (accumulate False) or added into."""
    import torch
    n_src, rows, d, stride = _src_geometry(src)
    T = rows - t_prev
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    _, _, _, dstride = _src_geometry(dsrc)
    dconv_w, dqueries, dgain, dmix_gain, dmix_w = grads
    if workspace is None:
        nbytes = msar_expand_bwd_workspace_size(n_src, T, d, src.dtype, ksizes)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=src.device)
    _check("msar_expand_bwd_chunk", load().msar_expand_bwd_chunk(
        _p(src), n_src, stride, t_prev, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries), _p(gain),
        eps, _p(mix_gain), _p(mix_w), mix_eps, _p(dh), _p(dsrc), dstride, 1 if accumulate else 0, _p(dconv_w),
        _p(dqueries), _p(dgain), _p(dmix_gain), _p(dmix_w), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return dsrc


@_on_stream
def msar_expand_fwd_ws(src, ksizes, conv_w, queries, gain=None, eps=1e-6, mix_gain=None, mix_w=None, mix_eps=1e-6,
                       out=None, workspace=None, stream=None):
    """MSAR read through the workspace chain.  conv_w: packed 1-D (shared
    kernels) or [n_src, stride] (each source's own) -> out [T, d]."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    m = queries.shape[0]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if out is None:
        out = torch.empty((T, d), dtype=src.dtype, device=src.device)
    if workspace is None:
        nbytes = msar_expand_fwd_ws_workspace_size(n_src, T, d, src.dtype)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=src.device)
    cstride = conv_w.stride(0) if conv_w.dim() == 2 else 0
    _check("msar_expand_fwd_ws", load().msar_expand_fwd_ws(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), cstride, _p(queries),
        _p(gain), eps, _p(mix_gain), _p(mix_w), mix_eps, _p(out), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def msar_block_phase1_ws_workspace_size(n_src, T, d, dtype, S):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    _check("msar_block_phase1_ws_workspace_size",
           load().msar_block_phase1_ws_workspace_size(n_src, T, d, dt, S, ctypes.byref(n)))
    return n.value


@_on_stream
def msar_block_phase1_ws(src, ksizes, conv_w, queries, gain=None, eps=1e-6, o=None, lse=None, workspace=None,
                         stream=None):
    """MSAR phase 1 through the workspace chain: queries [S, m, d] ->
    (o [S, m, T, d], lse [S, m, T])."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    S, m = queries.shape[0], queries.shape[1]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if o is None:
        o = torch.empty((S, m, T, d), dtype=src.dtype, device=src.device)
    if lse is None:
        lse = torch.empty((S, m, T), dtype=torch.float32, device=src.device)
    if workspace is None:
        nbytes = msar_block_phase1_ws_workspace_size(n_src, T, d, src.dtype, S)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=src.device)
    _check("msar_block_phase1_ws", load().msar_block_phase1_ws(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries), S, _p(gain), eps,
        _p(o), _p(lse), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return o, lse


def msar_block_phase2_ws_workspace_size(T, d, dtype):
    import torch
    n = ctypes.c_size_t(0)
    dt = BF16 if dtype == torch.bfloat16 else F32
    _check("msar_block_phase2_ws_workspace_size", load().msar_block_phase2_ws_workspace_size(T, d, dt, ctypes.byref(n)))
    return n.value


@_on_stream
def msar_block_phase2_ws(o, lse, partial, ksizes, conv_w, query, gain=None, eps=1e-6, mix_gain=None, mix_w=None,
                         mix_eps=1e-6, out=None, workspace=None, stream=None):
    """MSAR phase 2 of one layer through the workspace chain: o [m, T, d],
    lse [m, T], partial [T, d] or None, query [m, d] -> out [T, d]."""
    import torch
    m, T, d = o.shape
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    if out is None:
        out = torch.empty((T, d), dtype=o.dtype, device=o.device)
    if workspace is None:
        nbytes = msar_block_phase2_ws_workspace_size(T, d, o.dtype)
        workspace = torch.empty((max(nbytes, 16) + 3) // 4, dtype=torch.float32, device=o.device)
    _check("msar_block_phase2_ws", load().msar_block_phase2_ws(
        _p(o), _p(lse), _p(partial), T, d, _dt(o), m, ctypes.cast(ks, _vp), _p(conv_w), _p(query), _p(gain), eps,
        _p(mix_gain), _p(mix_w), mix_eps, _p(out), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


@_on_stream
def msar_block_phase2_bwd(o, lse, partial, ksizes, conv_w, query, dh, gain=None, eps=1e-6, mix_gain=None, mix_w=None,
                          mix_eps=1e-6, outs=None, workspace=None, stream=None):
    """Backward of msar_block_phase2 for dh [T, d] -> (d_o [m,T,d], d_lse
    [m,T], d_partial [T,d] or None, dconv_w, dquery [m,d], dgain [d],
    dmix_gain [m*d], dmix_w [m*d,m]).  outs: those eight tensors to write
    (else allocated here)."""
    import torch
    m, T, d = o.shape
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    dev, f32 = o.device, dict(dtype=torch.float32, device=o.device)
    if outs is not None:
        d_o, d_lse, d_p, dcw, dq, dg, dmg, dmw = outs
    else:
        d_o = torch.empty_like(o)
        d_lse = torch.empty((m, T), **f32)
        d_p = torch.empty_like(partial) if partial is not None else None
        dcw, dq, dg = torch.empty_like(conv_w, dtype=torch.float32), torch.empty((m, d), **f32), torch.empty((d,), **f32)
        dmg, dmw = torch.empty((m * d,), **f32), torch.empty((m * d, m), **f32)
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check("msar_block_phase2_bwd_workspace_size", load().msar_block_phase2_bwd_workspace_size(
            T, d, _dt(o), m, ctypes.cast(ks, _vp), ctypes.byref(n)))
        workspace = torch.empty((max(n.value, 16) + 3) // 4, dtype=torch.float32, device=dev)
    _check("msar_block_phase2_bwd", load().msar_block_phase2_bwd(
        _p(o), _p(lse), _p(partial), T, d, _dt(o), m, ctypes.cast(ks, _vp), _p(conv_w), _p(query), _p(gain), eps,
        _p(mix_gain), _p(mix_w), mix_eps, _p(dh), _p(d_o), _p(d_lse), _p(d_p), _p(dcw), _p(dq), _p(dg), _p(dmg),
        _p(dmw), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return d_o, d_lse, d_p, dcw, dq, dg, dmg, dmw


@_on_stream
def msar_block_phase1_bwd(src, ksizes, conv_w, queries, d_o, d_lse, gain=None, eps=1e-6, outs=None, workspace=None,
                          stream=None):
    """Backward of msar_block_phase1 for d_o [S,m,T,d], d_lse [S,m,T] ->
    (dsrc [n_src,T,d], dconv_w, dqueries [S,m,d], dgain [d]).  outs: those
    four tensors to write (else allocated here)."""
    import torch
    n_src, T, d, stride = _src_geometry(src)
    S, m = queries.shape[0], queries.shape[1]
    ks = (ctypes.c_int32 * len(ksizes))(*[int(k) for k in ksizes])
    dev, f32 = src.device, dict(dtype=torch.float32, device=src.device)
    if outs is not None:
        dsrc, dcw, dq, dg = outs
    else:
        dsrc = torch.empty((n_src, T, d), dtype=src.dtype, device=dev)
        dcw, dq, dg = (torch.empty_like(conv_w, dtype=torch.float32), torch.empty((S, m, d), **f32),
                       torch.empty((d,), **f32))
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check("msar_block_phase1_bwd_workspace_size", load().msar_block_phase1_bwd_workspace_size(
            n_src, T, d, _dt(src), m, ctypes.cast(ks, _vp), S, ctypes.byref(n)))
        workspace = torch.empty((max(n.value, 16) + 3) // 4, dtype=torch.float32, device=dev)
    _check("msar_block_phase1_bwd", load().msar_block_phase1_bwd(
        _p(src), n_src, stride, T, d, _dt(src), m, ctypes.cast(ks, _vp), _p(conv_w), _p(queries), S, _p(gain), eps,
        _p(d_o), _p(d_lse), _p(dsrc), T * d, _p(dcw), _p(dq), _p(dg), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return dsrc, dcw, dq, dg


# --------------------------------------------------------------------------
# The quantised depth cache, and phase 2 with the sublayer's norm in 8 bits
# --------------------------------------------------------------------------
# A decode step makes a few of these calls for every layer, and its kernels take
# a few microseconds: the checks below are kept to what the C side cannot see.

def _call(fn, dev, stream, *args):
    """Calls an entry point on device `dev`'s current stream (or `stream`), with that
    device current."""
    import torch
    f = getattr(load(), fn)
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status != OK:
        raise AttnResError(fn, status)


def _cuda(fn, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{fn}: a tensor on {t.device}; CUDA tensors are needed")
    return dev


def _is(fn, what, t, dev, dtype, shape):
    """t is a contiguous tensor of this device, dtype and shape: its pointer.  None passes."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {what} is {t.dtype}, {dtype} is needed")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {what} is on {t.device}, the other tensors on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {what} has shape {tuple(t.shape)}, {tuple(shape)} is needed")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {what} is not contiguous")
    return t.data_ptr()


def _blocks(fn, what, t, dev, shape):
    """t is an [n, T, width] tensor of this device and shape whose sources are
    contiguous blocks: the stride between them."""
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {what} is on {t.device}, the other tensors on cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {what} has shape {tuple(t.shape)}, {tuple(shape)} is needed")
    n, T, width = shape
    if t.is_contiguous():
        return T * width
    a, b, c = t.stride()
    if T and ((width > 1 and c != 1) or (T > 1 and b != width)):
        raise ValueError(f"{fn}: each source of {what} must be a contiguous block")
    # one source, or none of its rows: its stride says nothing
    return a if n > 1 and T else T * width


@functools.lru_cache(maxsize=None)
def attnres_cache_row_bytes(fmt, d, H=1):
    """Bytes of a row of the quantised cache."""
    n = ctypes.c_size_t(0)
    _check("attnres_cache_row_bytes", load().attnres_cache_row_bytes(fmt, d, H, ctypes.byref(n)))
    return n.value


def _rows(fn, cache):
    import torch
    if cache.dtype is not torch.uint8 or cache.dim() != 3:
        raise TypeError(f"{fn}: the cache is uint8 [n_src, T, row_bytes]")
    return _cuda(fn, cache)


@_on_stream
def attnres_cache_quant(src, fmt, H=1, f=None, cache=None, stream=None):
    """Quantise src [n_src,T,d] (plus f, like src) into cache rows: cache uint8
    [n_src,T,row_bytes], allocated here unless given (sources may be strided)."""
    fn = "attnres_cache_quant"
    if src.dim() != 3:
        raise ValueError(f"{fn}: src is [n_src, T, d]")
    dev = _cuda(fn, src)
    n_src, T, d = shape = src.shape
    stride = _blocks(fn, "src", src, dev, shape)
    if f is not None and (f.dtype is not src.dtype or _blocks(fn, "f", f, dev, shape) != stride):
        raise ValueError(f"{fn}: f must be like src, strides included")
    rows = (n_src, T, attnres_cache_row_bytes(fmt, d, H))
    if cache is None:
        import torch
        cache = torch.empty(rows, dtype=torch.uint8, device=src.device)
    else:
        _rows(fn, cache)
    _call(fn, dev, stream, src.data_ptr(), None if f is None else f.data_ptr(), n_src, stride, T, d, H, _dt(src), fmt,
          cache.data_ptr(), _blocks(fn, "cache", cache, dev, rows))
    return cache


@_on_stream
def attnres_cache_dequant(cache, fmt, d, H=1, dtype=None, out=None, stream=None):
    """Values of cache rows [n_src,T,row_bytes] as dtype (bfloat16) -> [n_src,T,d]."""
    fn = "attnres_cache_dequant"
    dev = _rows(fn, cache)
    n_src, T, _ = cache.shape
    cstride = _blocks(fn, "cache", cache, dev, (n_src, T, attnres_cache_row_bytes(fmt, d, H)))
    if out is None:
        import torch
        out = torch.empty((n_src, T, d), dtype=dtype or torch.bfloat16, device=cache.device)
    elif dtype is not None and out.dtype is not dtype:
        raise TypeError(f"{fn}: out is {out.dtype}, {dtype} was asked for")
    _call(fn, dev, stream, cache.data_ptr(), n_src, cstride, T, d, H, fmt, _dt(out), out.data_ptr(),
          _blocks(fn, "out", out, dev, (n_src, T, d)))
    return out


@_on_stream
def attnres_cache_read(cache, fmt, queries, gain=None, eps=1e-6, dtype=None, out=None, lse=None, want_lse=True,
                       stream=None):
    """The depth read over a quantised cache [n_src,T,row_bytes]: queries [n_q,d]
    -> (out [n_q,T,d], lse [n_q,T]); queries [n_q,H,d/H] (MHAR) -> lse [n_q,H,T]."""
    import torch
    fn = "attnres_cache_read"
    f32 = torch.float32
    dev = _rows(fn, cache)
    n_src, T, _ = cache.shape
    qshape = queries.shape
    if len(qshape) == 2:
        (n_q, d), H = qshape, 1
        lshape = (n_q, T)
    elif len(qshape) == 3:
        n_q, H, d = qshape
        d *= H
        lshape = (n_q, H, T)
    else:
        raise ValueError(f"{fn}: queries are [n_q, d] or [n_q, H, d/H]")
    cstride = _blocks(fn, "cache", cache, dev, (n_src, T, attnres_cache_row_bytes(fmt, d, H)))
    if out is None:
        out = torch.empty((n_q, T, d), dtype=dtype or torch.bfloat16, device=cache.device)
    else:
        _is(fn, "out", out, dev, dtype or out.dtype, (n_q, T, d))
    if lse is None:
        if want_lse:
            lse = torch.empty(lshape, dtype=f32, device=cache.device)
    else:
        _is(fn, "lse", lse, dev, f32, lshape)
    _call(fn, dev, stream, cache.data_ptr(), n_src, cstride, T, d, H, fmt, _is(fn, "queries", queries, dev, f32, qshape),
          n_q, _is(fn, "gain", gain, dev, f32, (d,)), eps, _dt(out), out.data_ptr(), None if lse is None else lse.data_ptr())
    return out, lse


Phase2Norm = collections.namedtuple("Phase2Norm", "codes scales partial h")


@_on_stream
def attnres_phase2_norm_q8(o, lse, partial, query, norm_gain=None, f=None, gain=None, eps=1e-6, norm_eps=1e-6, group=0,
                           partial_out=None, want_h=False, h=None, codes=None, scales=None, stream=None):
    """Phase 2 and the sublayer's RMSNorm in 8 bits: o [T,d], lse [T] or [H,T],
    partial [T,d], f [T,d], each may be None (o None: a plain residual layer;
    partial and f None: a block's first layer); query [d], or [H,d/H] for heads.
    -> Phase2Norm(codes float8_e4m3fn [T,d], scales [T, d/group or 1], partial
    (partial + f when f is given), h (or None))."""
    import torch
    fn = "attnres_phase2_norm_q8"
    f32 = torch.float32
    ref = o if o is not None else partial if partial is not None else f
    if ref is None:
        raise ValueError(f"{fn}: o, partial and f are all None")
    shape = ref.shape
    if len(shape) != 2:
        raise ValueError(f"{fn}: o, partial and f are [T, d]")
    T, d = shape
    dt, dev, device = ref.dtype, _cuda(fn, ref), ref.device
    if group and (group < 0 or d % group):
        raise ValueError(f"{fn}: {d} channels are not whole groups of {group}")
    H, p_lse, p_query, p_gain = 1, None, None, None
    if o is not None and (partial is not None or f is not None):
        if query is None or lse is None:
            raise ValueError(f"{fn}: a merge needs lse and query")
        if query.dim() == 2:
            H = query.shape[0]
            p_query, p_lse = _is(fn, "query", query, dev, f32, (H, d // H)), _is(fn, "lse", lse, dev, f32, (H, T))
        else:
            p_query, p_lse = _is(fn, "query", query, dev, f32, (d,)), _is(fn, "lse", lse, dev, f32, (T,))
        p_gain = _is(fn, "gain", gain, dev, f32, (d,))
    p_o, p_partial, p_f = (_is(fn, "o", o, dev, dt, shape), _is(fn, "partial", partial, dev, dt, shape),
                           _is(fn, "f", f, dev, dt, shape))
    if f is None:
        partial_out, p_out = None, None
    elif partial_out is None:
        partial_out = torch.empty_like(f)
        p_out = partial_out.data_ptr()
    else:
        p_out = _is(fn, "partial_out", partial_out, dev, dt, shape)
    if h is None:
        if want_h:
            h = torch.empty_like(ref)
    else:
        _is(fn, "h", h, dev, dt, shape)
    if codes is None:
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=device)
    else:
        _is(fn, "codes", codes, dev, torch.float8_e4m3fn, shape)
    groups = (T, d // group if group else 1)
    if scales is None:
        scales = torch.empty(groups, dtype=f32, device=device)
    else:
        _is(fn, "scales", scales, dev, f32, groups)
    _call(fn, dev, stream, p_o, p_lse, p_partial, p_f, p_out, T, d, H, _dt(ref), p_query, p_gain, eps,
          _is(fn, "norm_gain", norm_gain, dev, f32, (d,)), norm_eps, group, codes.data_ptr(), scales.data_ptr(),
          None if h is None else h.data_ptr())
    return Phase2Norm(codes, scales, partial if f is None else partial_out, h)


@functools.lru_cache(maxsize=1024)
def _norm_bwd_workspace_size(T, d, dt, dev):
    n = ctypes.c_size_t(0)
    _check("attnres_norm_bwd_workspace_size", load().attnres_norm_bwd_workspace_size(T, d, dt, ctypes.byref(n)))
    return n.value


def attnres_norm_bwd_workspace_size(T, d, dtype):
    """Bytes on the current device."""
    import torch
    return _norm_bwd_workspace_size(T, d, BF16 if dtype == torch.bfloat16 else F32, torch.cuda.current_device())


@_on_stream
def attnres_norm_bwd(h, dy, gain=None, eps=1e-6, dres=None, dh=None, dgain=None, workspace=None, stream=None):
    """Backward of the sublayer's RMSNorm for h, dy [T,d] (dres [T,d]: the gradient
    past the norm) -> (dh [T,d], dgain [d]).  The workspace is allocated here
    unless given."""
    import torch
    fn = "attnres_norm_bwd"
    f32 = torch.float32
    shape = h.shape
    if len(shape) != 2:
        raise ValueError(f"{fn}: h is [T, d]")
    T, d = shape
    dt, dev, device = h.dtype, _cuda(fn, h), h.device
    p_h, p_dy, p_dres = (_is(fn, "h", h, dev, dt, shape), _is(fn, "dy", dy, dev, dt, shape),
                         _is(fn, "dres", dres, dev, dt, shape))
    p_gain = _is(fn, "gain", gain, dev, f32, (d,))
    if dh is None:
        dh = torch.empty_like(h)
    else:
        _is(fn, "dh", dh, dev, dt, shape)
    if dgain is None:
        dgain = torch.empty((d,), dtype=f32, device=device)
    else:
        _is(fn, "dgain", dgain, dev, f32, (d,))
    if workspace is None:
        with torch.cuda.device(dev) if dev != torch._C._cuda_getDevice() else contextlib.nullcontext():
            nbytes = _norm_bwd_workspace_size(T, d, _dt(h), dev)
        workspace = torch.empty(((max(nbytes, 16) + 3) // 4,), dtype=f32, device=device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{fn}: the workspace must be contiguous, on cuda:{dev}")
    _call(fn, dev, stream, p_h, p_dy, p_dres, T, d, _dt(h), p_gain, eps, dh.data_ptr(), dgain.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dh, dgain
