"""Python binding of libgdr (ctypes).  Argument marshalling only: every step of
the recurrence runs in the library's CUDA kernels.

The functions carry the C ABI's names (include/gdr.h) and take torch CUDA
tensors; they check dtype, device and contiguity, pass raw pointers and the
current CUDA stream, and raise ``GdrError`` on any non-OK status.  There is no
fallback: if libgdr.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr.so")

GDR_OK = 0
GDR_ERR_INVALID_ARG = 1
GDR_ERR_UNSUPPORTED = 2
GDR_ERR_WORKSPACE = 3
GDR_ERR_CUDA = 4
GDR_ERR_DEVICE_TIMEOUT = 5

GDR_GATE_SCALAR = 0
GDR_GATE_CHANNEL = 1
GDR_F32 = 0
GDR_BF16 = 1
GDR_PATH_SIMT = 0
GDR_PATH_TCGEN05 = 1
GDR_PATH_TCGEN05_SPLIT = 2
GDR_PROLOGUE_SILU = 1
GDR_PROLOGUE_NORMALIZE_QK = 2
GDR_ACT_NONE = 0
GDR_ACT_SILU = 1
GDR_ACT_SIGMOID = 2

# Every symbol include/gdr.h declares.
EXPORTED = ("gdr_status_string", "gdr_prefill_workspace_size", "gdr_prefill_path",
            "gdr_prefill_chunked", "gdr_prefill_check_workspace", "gdr_decode_step",
            "gdr_prefill_chunked_noalloc", "gdr_prefill_chunked_gqa", "gdr_decode_step_gqa",
            "gdr_decode_multi", "gdr_prefill_plan", "gdr_prologue", "gdr_backward",
            "gdr_backward_workspace_size", "gdr_prefill_noalloc_check",
            "gdr_test_noalloc_wait_timeout", "gdr_prefill_fused", "gdr_linear_workspace_size",
            "gdr_linear_prefill", "gdr_linear_decode", "gdr_linear_backward",
            "gdr_linear_check_workspace", "gdr_norm_gate", "gdr_norm_gate_workspace_size",
            "gdr_norm_gate_backward")


class GdrError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdr_status_string(status)}")


_lock = threading.Lock()
_lib = None


def load_library():
    """Load libgdr.so once (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgdr.so not built ({LIB_PATH}); run "
                               "`python -m gated_delta_rule_151_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        ST = ctypes.c_int
        lib.gdr_status_string.argtypes = [ST]
        lib.gdr_status_string.restype = ctypes.c_char_p
        lib.gdr_prefill_workspace_size.argtypes = [I32, I32, I32, I32, I32, ST, ST,
                                                   ctypes.POINTER(SZ)]
        lib.gdr_prefill_workspace_size.restype = ST
        lib.gdr_prefill_path.argtypes = [I32, I32, ST, ST, ctypes.POINTER(ctypes.c_int)]
        lib.gdr_prefill_path.restype = ST
        lib.gdr_prefill_plan.argtypes = [I32, I32, I32, I32, I32, ST, ST, SZ,
                                         ctypes.POINTER(ctypes.c_int)]
        lib.gdr_prefill_plan.restype = ST
        lib.gdr_prefill_chunked.argtypes = [P, P, P, P, P, P, P, I32, I32, I32, I32, I32, ST, ST,
                                            P, P, P, SZ, P]
        lib.gdr_prefill_chunked.restype = ST
        lib.gdr_prefill_check_workspace.argtypes = [P, SZ, P]
        lib.gdr_prefill_check_workspace.restype = ST
        lib.gdr_decode_step.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, ST, ST, P, P]
        lib.gdr_decode_step.restype = ST
        lib.gdr_prefill_chunked_noalloc.argtypes = [P, P, P, P, P, P, P, I32, I32, I32, I32, I32,
                                                    ST, ST, P, P, P]
        lib.gdr_prefill_chunked_noalloc.restype = ST
        lib.gdr_prefill_noalloc_check.argtypes = [P]
        lib.gdr_prefill_noalloc_check.restype = ST
        lib.gdr_test_noalloc_wait_timeout.argtypes = [ctypes.c_uint32, P]
        lib.gdr_test_noalloc_wait_timeout.restype = ST
        lib.gdr_prefill_chunked_gqa.argtypes = [P, P, P, P, P, P, P, I32, I32, I32, I32, I32, I32,
                                                ST, ST, P, P, P, SZ, P]
        lib.gdr_prefill_chunked_gqa.restype = ST
        lib.gdr_decode_step_gqa.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, ST, ST, P, P]
        lib.gdr_decode_step_gqa.restype = ST
        lib.gdr_decode_multi.argtypes = [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, ST, ST, P,
                                         P, P]
        lib.gdr_decode_multi.restype = ST
        lib.gdr_prologue.argtypes = [P] * 12 + [I32] * 6 + [ST, ST, ctypes.c_uint32] + [P] * 6
        lib.gdr_prologue.restype = ST
        lib.gdr_prefill_fused.argtypes = ([P] * 13 + [I32] * 6 + [ST, ST, ctypes.c_uint32] +
                                          [P, P, P, SZ, P])
        lib.gdr_prefill_fused.restype = ST
        lib.gdr_backward_workspace_size.argtypes = [I32, I32, I32, I32, I32, ctypes.POINTER(SZ)]
        lib.gdr_backward_workspace_size.restype = ST
        lib.gdr_backward.argtypes = [P] * 7 + [I32] * 6 + [ST, ST] + [P] * 9 + [SZ, P]
        lib.gdr_backward.restype = ST
        I64, F32 = ctypes.c_int64, ctypes.c_float
        lib.gdr_linear_workspace_size.argtypes = [I32] * 6 + [ST, I32, ctypes.POINTER(SZ)]
        lib.gdr_linear_workspace_size.restype = ST
        lib.gdr_linear_prefill.argtypes = [P] * 6 + [I32] * 6 + [ST, P, P, P, SZ, P]
        lib.gdr_linear_prefill.restype = ST
        lib.gdr_linear_decode.argtypes = [P] * 5 + [I32] * 5 + [ST, P, P]
        lib.gdr_linear_decode.restype = ST
        lib.gdr_linear_backward.argtypes = [P] * 6 + [I32] * 6 + [ST] + [P] * 7 + [SZ, P]
        lib.gdr_linear_backward.restype = ST
        lib.gdr_linear_check_workspace.argtypes = [P, SZ, P]
        lib.gdr_linear_check_workspace.restype = ST
        lib.gdr_norm_gate.argtypes = [P] * 5 + [I64, I32, F32, F32, ST, ST, P, P, P]
        lib.gdr_norm_gate.restype = ST
        lib.gdr_norm_gate_workspace_size.argtypes = [I64, I32, ctypes.POINTER(SZ)]
        lib.gdr_norm_gate_workspace_size.restype = ST
        lib.gdr_norm_gate_backward.argtypes = ([P] * 5 + [I64, I32, F32, F32, ST, ST] + [P] * 8 +
                                               [SZ, P])
        lib.gdr_norm_gate_backward.restype = ST
        _lib = lib
        return lib


def gdr_status_string(status: int) -> str:
    return load_library().gdr_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != GDR_OK:
        raise GdrError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return GDR_BF16
    if dtype == torch.float32:
        return GDR_F32
    raise TypeError(f"io dtype must be bfloat16 or float32, got {dtype}")


def _need(t, name, dtype=None, ndim=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def gdr_prefill_workspace_size(num_seqs, total_T, H, d_k, d_v, gate_mode, io_dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().gdr_prefill_workspace_size(num_seqs, total_T, H, d_k, d_v, gate_mode,
                                                     io_dtype, ctypes.byref(out)),
           "gdr_prefill_workspace_size")
    return int(out.value)


def gdr_prefill_path(d_k, d_v, gate_mode, io_dtype) -> int:
    out = ctypes.c_int(0)
    _check(load_library().gdr_prefill_path(d_k, d_v, gate_mode, io_dtype, ctypes.byref(out)),
           "gdr_prefill_path")
    return int(out.value)


def gdr_prefill_plan(num_seqs, total_T, H, d_k, d_v, gate_mode, io_dtype,
                     workspace_bytes) -> int:
    """The plan gdr_prefill_chunked runs with this much workspace:
    GDR_PATH_SIMT, GDR_PATH_TCGEN05 or GDR_PATH_TCGEN05_SPLIT."""
    out = ctypes.c_int(0)
    _check(load_library().gdr_prefill_plan(num_seqs, total_T, H, d_k, d_v, gate_mode, io_dtype,
                                           workspace_bytes, ctypes.byref(out)),
           "gdr_prefill_plan")
    return int(out.value)


def _prefill(name, q, k, v, g, beta, initial_state, cu_seqlens, num_seqs, o, final_state,
             output_final_state, workspace, stream):
    _need(q, "q", ndim=3)
    io = q.dtype
    _need(k, "k", io, 3)
    _need(v, "v", io, 3)
    _need(beta, "beta", torch.float32, 2)
    _need(g, "g", torch.float32)
    T, Hqk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    if g.dim() == 2:
        gate = GDR_GATE_SCALAR
    elif g.dim() == 3:
        gate = GDR_GATE_CHANNEL
    else:
        raise ValueError("g must be [T, H] or [T, H, d_k]")
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, 4)
    if o is None:
        o = torch.empty((T, H, dv), dtype=io, device=q.device)
    _need(o, "o", io, 3)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, 4)
    io_code = _io_code(io)
    ws_bytes = gdr_prefill_workspace_size(N, T, H, dk, dv, gate, io_code)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    lib = load_library()
    heads = (Hqk, H) if name == "gdr_prefill_chunked_gqa" else (H,)
    if name == "gdr_prefill_chunked" and Hqk != H:
        raise ValueError("q/k and v head counts differ: use gdr_prefill_chunked_gqa")
    st = getattr(lib, name)(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
        N, T, *heads, dk, dv, gate, io_code, _ptr(o), _ptr(final_state), _ptr(workspace),
        workspace.numel() if workspace is not None else 0, _stream_ptr(stream))
    _check(st, name)
    return o, final_state


def gdr_prefill_chunked(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *,
                        num_seqs=None, o=None, final_state=None, output_final_state=True,
                        workspace=None, stream=None):
    """Chunked prefill (see include/gdr.h).  Returns (o, final_state).

    q, k [T, H, d_k], v [T, H, d_v] (bf16 or fp32); g [T, H] or [T, H, d_k]
    fp32; beta [T, H] fp32; initial_state [N, H, d_v, d_k] fp32 or None;
    cu_seqlens int32 [N + 1] on the device, or None with ``num_seqs`` equal
    sequences (default 1).  ``final_state`` may be given (it may be the same
    tensor as initial_state); otherwise one is allocated when
    ``output_final_state``.
    """
    return _prefill("gdr_prefill_chunked", q, k, v, g, beta, initial_state, cu_seqlens, num_seqs,
                    o, final_state, output_final_state, workspace, stream)


def gdr_prefill_chunked_gqa(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *,
                            num_seqs=None, o=None, final_state=None, output_final_state=True,
                            workspace=None, stream=None):
    """Chunked prefill with grouped query/key heads: q, k [T, H_qk, d_k],
    everything else per value head [T, H, ...]; H_qk divides H."""
    return _prefill("gdr_prefill_chunked_gqa", q, k, v, g, beta, initial_state, cu_seqlens,
                    num_seqs, o, final_state, output_final_state, workspace, stream)


def gdr_prefill_check_workspace(workspace, stream=None):
    _check(load_library().gdr_prefill_check_workspace(
        _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream_ptr(stream)),
        "gdr_prefill_check_workspace")


def _decode(name, q, k, v, g, beta, state, o, stream):
    _need(q, "q", ndim=3)
    io = q.dtype
    _need(k, "k", io, 3)
    _need(v, "v", io, 3)
    _need(beta, "beta", torch.float32, 2)
    _need(g, "g", torch.float32)
    _need(state, "state", torch.float32, 4)
    N, Hqk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    gate = GDR_GATE_SCALAR if g.dim() == 2 else GDR_GATE_CHANNEL
    if o is None:
        o = torch.empty((N, H, dv), dtype=io, device=q.device)
    _need(o, "o", io, 3)
    if name == "gdr_decode_step" and Hqk != H:
        raise ValueError("q/k and v head counts differ: use gdr_decode_step_gqa")
    heads = (Hqk, H) if name == "gdr_decode_step_gqa" else (H,)
    st = getattr(load_library(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                       _ptr(state), N, *heads, dk, dv, gate, _io_code(io), _ptr(o),
                                       _stream_ptr(stream))
    _check(st, name)
    return o


def gdr_decode_step(q, k, v, g, beta, state, *, o=None, stream=None):
    """One decode step (see include/gdr.h): state is updated in place.

    q, k [N, H, d_k], v [N, H, d_v] (bf16 or fp32); g [N, H] or [N, H, d_k]
    fp32; beta [N, H] fp32; state [N, H, d_v, d_k] fp32.  Returns o [N, H, d_v].
    """
    return _decode("gdr_decode_step", q, k, v, g, beta, state, o, stream)


def gdr_decode_step_gqa(q, k, v, g, beta, state, *, o=None, stream=None):
    """One decode step with grouped query/key heads: q, k [N, H_qk, d_k]."""
    return _decode("gdr_decode_step_gqa", q, k, v, g, beta, state, o, stream)


def gdr_prefill_chunked_noalloc(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *,
                                num_seqs=None, o=None, final_state=None, stream=None):
    """gdr_prefill_chunked without a workspace: the library's own fixed device
    scratch is used instead (see include/gdr.h for who needs this and the
    rules that come with it).  ``o`` must be given; ``final_state`` is
    optional (None: the final state is not written, and None is returned for
    it).  gdr_prefill_noalloc_check reports a device-side wait that gave up."""
    _need(q, "q", ndim=3)
    io = q.dtype
    _need(k, "k", io, 3)
    _need(v, "v", io, 3)
    _need(beta, "beta", torch.float32, 2)
    _need(g, "g", torch.float32)
    _need(o, "o", io, 3)
    T, H, dk = q.shape
    dv = v.shape[2]
    gate = GDR_GATE_SCALAR if g.dim() == 2 else GDR_GATE_CHANNEL
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, 4)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, 4)
    st = load_library().gdr_prefill_chunked_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
        N, T, H, dk, dv, gate, _io_code(io), _ptr(o), _ptr(final_state), _stream_ptr(stream))
    _check(st, "gdr_prefill_chunked_noalloc")
    return o, final_state


def gdr_prefill_noalloc_check(stream=None):
    """Raise GdrError(GDR_ERR_DEVICE_TIMEOUT) if a bounded device-side wait of
    a no-alloc prefill gave up since the previous check (synchronises the
    stream; the error word is cleared once read)."""
    _check(load_library().gdr_prefill_noalloc_check(_stream_ptr(stream)),
           "gdr_prefill_noalloc_check")


def gdr_decode_multi(q, k, v, g, beta, state, *, o=None, snapshots=None, stream=None):
    """T consecutive decode steps per sequence in one pass (see include/gdr.h).

    q, k [N, T, H_qk, d_k]; v [N, T, H, d_v]; g [N, T, H] or [N, T, H, d_k];
    beta [N, T, H]; state [N, H, d_v, d_k] updated in place; optional
    snapshots [N, T, H, d_v, d_k] receive the state after every token.
    Returns o [N, T, H, d_v].
    """
    _need(q, "q", ndim=4)
    io = q.dtype
    _need(k, "k", io, 4)
    _need(v, "v", io, 4)
    _need(beta, "beta", torch.float32, 3)
    _need(g, "g", torch.float32)
    _need(state, "state", torch.float32, 4)
    N, T, Hqk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    gate = GDR_GATE_SCALAR if g.dim() == 3 else GDR_GATE_CHANNEL
    if o is None:
        o = torch.empty((N, T, H, dv), dtype=io, device=q.device)
    _need(o, "o", io, 4)
    if snapshots is not None:
        _need(snapshots, "snapshots", torch.float32, 5)
    st = load_library().gdr_decode_multi(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                         _ptr(state), N, T, Hqk, H, dk, dv, gate, _io_code(io),
                                         _ptr(o), _ptr(snapshots), _stream_ptr(stream))
    _check(st, "gdr_decode_multi")
    return o


def gdr_prologue(xq, xk, xv, wq, wk, wv, xg, gscale, xb, conv_state_in=None, cu_seqlens=None, *,
                 num_seqs=None, conv_state_out=None, silu=False, normalize_qk=True, q=None,
                 k=None, v=None, g=None, beta=None, stream=None):
    """Input-side prologue (see include/gdr.h): short causal convolution with
    state, optional SiLU, q/k L2 normalisation, beta and log-gate maps.

    xq, xk [T, H_qk, d_k]; xv [T, H, d_v] (bf16 or fp32); wq, wk [H_qk d_k, 4];
    wv [H d_v, 4]; xg [T, H] or [T, H, d_k]; gscale [H]; xb [T, H];
    conv_state_in / conv_state_out [N, 2 H_qk d_k + H d_v, 3] fp32 or None.
    Returns (q, k, v, g, beta).
    """
    _need(xq, "xq", ndim=3)
    io = xq.dtype
    _need(xk, "xk", io, 3)
    _need(xv, "xv", io, 3)
    for t, name in ((wq, "wq"), (wk, "wk"), (wv, "wv")):
        _need(t, name, torch.float32, 2)
    _need(xg, "xg", torch.float32)
    _need(gscale, "gscale", torch.float32, 1)
    _need(xb, "xb", torch.float32, 2)
    T, Hqk, dk = xq.shape
    H, dv = xv.shape[1], xv.shape[2]
    gate = GDR_GATE_SCALAR if xg.dim() == 2 else GDR_GATE_CHANNEL
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n = cu_seqlens.numel() - 1
    else:
        n = 1 if num_seqs is None else int(num_seqs)
    if conv_state_in is not None:
        _need(conv_state_in, "conv_state_in", torch.float32, 3)
    if conv_state_out is not None:
        _need(conv_state_out, "conv_state_out", torch.float32, 3)
    dev = xq.device
    q = torch.empty_like(xq) if q is None else q
    k = torch.empty_like(xk) if k is None else k
    v = torch.empty_like(xv) if v is None else v
    g = torch.empty(xg.shape, dtype=torch.float32, device=dev) if g is None else g
    beta = torch.empty(xb.shape, dtype=torch.float32, device=dev) if beta is None else beta
    flags = (GDR_PROLOGUE_SILU if silu else 0) | (GDR_PROLOGUE_NORMALIZE_QK if normalize_qk else 0)
    st = load_library().gdr_prologue(
        _ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(xg), _ptr(gscale),
        _ptr(xb), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(cu_seqlens), n, T, Hqk, H, dk,
        dv, gate, _io_code(io), flags, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
        _stream_ptr(stream))
    _check(st, "gdr_prologue")
    return q, k, v, g, beta


def gdr_prefill_fused(xq, xk, xv, wq, wk, wv, xg, gscale, xb, conv_state_in=None,
                      initial_state=None, cu_seqlens=None, *, num_seqs=None, conv_state_out=None,
                      silu=False, normalize_qk=True, o=None, final_state=None,
                      output_final_state=True, workspace=None, stream=None):
    """The prologue fused into the chunked prefill (see include/gdr.h):
    raw inputs as for gdr_prologue, the state and outputs as for
    gdr_prefill_chunked_gqa.  Returns (o, final_state)."""
    _need(xq, "xq", torch.bfloat16, 3)
    _need(xk, "xk", torch.bfloat16, 3)
    _need(xv, "xv", torch.bfloat16, 3)
    for t, name in ((wq, "wq"), (wk, "wk"), (wv, "wv")):
        _need(t, name, torch.float32, 2)
    _need(xg, "xg", torch.float32)
    _need(gscale, "gscale", torch.float32, 1)
    _need(xb, "xb", torch.float32, 2)
    T, Hqk, dk = xq.shape
    H, dv = xv.shape[1], xv.shape[2]
    gate = GDR_GATE_SCALAR if xg.dim() == 2 else GDR_GATE_CHANNEL
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
        N = cu_seqlens.numel() - 1
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    for t, name in ((conv_state_in, "conv_state_in"), (conv_state_out, "conv_state_out")):
        if t is not None:
            _need(t, name, torch.float32, 3)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, 4)
    dev = xq.device
    if o is None:
        o = torch.empty((T, H, dv), dtype=torch.bfloat16, device=dev)
    _need(o, "o", torch.bfloat16, 3)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    if final_state is not None:
        _need(final_state, "final_state", torch.float32, 4)
    ws_bytes = gdr_prefill_workspace_size(N, T, H, dk, dv, gate, GDR_BF16)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    flags = (GDR_PROLOGUE_SILU if silu else 0) | (GDR_PROLOGUE_NORMALIZE_QK if normalize_qk else 0)
    st = load_library().gdr_prefill_fused(
        _ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(xg), _ptr(gscale),
        _ptr(xb), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(initial_state),
        _ptr(cu_seqlens), N, T, Hqk, H, dk, dv, gate, GDR_BF16, flags, _ptr(o),
        _ptr(final_state), _ptr(workspace), workspace.numel() if workspace is not None else 0,
        _stream_ptr(stream))
    _check(st, "gdr_prefill_fused")
    return o, final_state


def gdr_backward_workspace_size(num_seqs, total_T, H, d_k, d_v) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().gdr_backward_workspace_size(num_seqs, total_T, H, d_k, d_v,
                                                      ctypes.byref(n)),
           "gdr_backward_workspace_size")
    return int(n.value)


def gdr_backward(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, d_o,
                 d_final_state=None, num_seqs=None, want_d_initial_state=True, workspace=None,
                 stream=None):
    """Gradient of <d_o, o> + <d_final_state, final_state> (see include/gdr.h).

    Inputs as for gdr_prefill_chunked_gqa; d_o [T, H, d_v] in the io dtype;
    d_final_state [N, H, d_v, d_k] fp32 or None.  Returns (dq, dk, dv, dg,
    dbeta, d_initial_state) as fp32 tensors (the last None unless wanted).
    Without a workspace one of gdr_backward_workspace_size bytes is
    allocated, which selects the chunked form where it applies (scalar gate,
    d = 128); a workspace too small for its records selects the per-token
    form.
    """
    _need(q, "q", ndim=3)
    io = q.dtype
    _need(k, "k", io, 3)
    _need(v, "v", io, 3)
    _need(d_o, "d_o", io, 3)
    _need(beta, "beta", torch.float32, 2)
    _need(g, "g", torch.float32)
    T, Hqk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    gate = GDR_GATE_SCALAR if g.dim() == 2 else GDR_GATE_CHANNEL
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, 1)
        n = cu_seqlens.numel() - 1
    else:
        n = 1 if num_seqs is None else int(num_seqs)
    if initial_state is not None:
        _need(initial_state, "initial_state", torch.float32, 4)
    if d_final_state is not None:
        _need(d_final_state, "d_final_state", torch.float32, 4)
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((T, Hqk, dk), **f32)
    dk_ = torch.empty((T, Hqk, dk), **f32)
    dv_ = torch.empty((T, H, dv), **f32)
    dg = torch.empty(g.shape, **f32)
    db = torch.empty((T, H), **f32)
    dh0 = torch.empty((n, H, dv, dk), **f32) if want_d_initial_state else None
    need = gdr_backward_workspace_size(n, T, H, dk, dv)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().gdr_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
        n, T, Hqk, H, dk, dv, gate, _io_code(io), _ptr(d_o), _ptr(d_final_state), _ptr(dq),
        _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(db), _ptr(dh0), _ptr(workspace), wsb,
        _stream_ptr(stream))
    _check(st, "gdr_backward")
    return dq, dk_, dv_, dg, db, dh0


# ---- linear attention with a decay for each head, and the norms around a block ----
#
# These calls run on the device of their first argument, whichever device is
# current, and allocate what the caller does not give under the stream they run
# on, so that the memory is not handed out again while a kernel still uses it.

_ACTIVATIONS = {"none": GDR_ACT_NONE, "silu": GDR_ACT_SILU, "sigmoid": GDR_ACT_SIGMOID}


# The handle of a device's current stream: 0.2 us by torch's own shortcut, where it
# has one, against 3 us for a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, stream, run):
    """run(handle of the stream), with ``device`` and ``stream`` current."""
    if stream is None and device.index == torch.cuda.current_device():
        return run(_raw_stream(device.index))
    if stream is not None and not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.device(device):
        if stream is None:
            return run(torch.cuda.current_stream().cuda_stream)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream)
        with torch.cuda.stream(stream):
            return run(stream.cuda_stream)


def _given(t, name, shape, dtype, device):
    """One tensor argument: on the device, contiguous, of this type and shape."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _int32(n, name):
    """n, which ctypes would otherwise cut to 32 bits."""
    if not -(1 << 31) <= n < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {n}")
    return n


def _at(t):
    return None if t is None else t.data_ptr()


def _scratch(workspace, need, like, device):
    """(pointer, bytes) of the caller's workspace or of a new one, and what keeps it alive.
    ``like``: an fp32 tensor of the call (its new_empty takes half of torch.empty's time)."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = like.new_empty((need + 3) // 4)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _linear_args(q, k, v, decay, cu_seqlens, num_seqs):
    """Checks what the linear-attention calls share; returns their sizes."""
    _need(q, "q", ndim=3)
    shape, dev, io = q.shape, q.device, q.dtype
    T, Hqk, dk = shape
    _given(k, "k", shape, io, dev)
    if v is None or v.dim() != 3:
        raise ValueError("v must be [T, H, d_v]")
    _, H, dv = v.shape
    _given(v, "v", (T, H, dv), io, dev)
    _given(decay, "decay", (H,), torch.float32, dev)
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if N < 0:
            raise ValueError("cu_seqlens must be [N + 1]")
        _given(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
        if num_seqs is not None and int(num_seqs) != N:
            raise ValueError(f"num_seqs is {num_seqs}, cu_seqlens has {N} sequences")
    else:
        N = 1 if num_seqs is None else int(num_seqs)
    if max(T, Hqk, H, dk, dv, abs(N)) >= 1 << 31:      # (ctypes would cut them to 32 bits)
        raise ValueError(f"sizes must fit 32 bits, got T {T}, heads {Hqk} and {H}, d {dk} and {dv}, {N} sequences")
    return T, Hqk, H, dk, dv, N, dev, io


@functools.lru_cache(maxsize=1024)
def _linear_bytes(*shape):
    n = ctypes.c_size_t(0)
    _check(load_library().gdr_linear_workspace_size(*shape, ctypes.byref(n)),
           "gdr_linear_workspace_size")
    return int(n.value)


def gdr_linear_workspace_size(num_seqs, total_T, H_qk, H, d_k, d_v, io_dtype,
                              backward=False) -> int:
    for n, name in ((num_seqs, "num_seqs"), (total_T, "total_T"), (H_qk, "H_qk"), (H, "H"), (d_k, "d_k"),
                    (d_v, "d_v")):
        _int32(n, name)
    return _linear_bytes(num_seqs, total_T, H_qk, H, d_k, d_v, io_dtype, int(backward))


def gdr_linear_prefill(q, k, v, decay, initial_state=None, cu_seqlens=None, *, num_seqs=None,
                       o=None, final_state=None, output_final_state=True, workspace=None,
                       stream=None):
    """Linear attention with a decay for each head over whole prompts (see
    include/gdr.h).  Returns (o, final_state).

    q, k [T, H_qk, d_k], v [T, H, d_v] (bf16 or fp32; H_qk divides H); decay
    [H] fp32, the log-decays; initial_state [N, H, d_v, d_k] fp32 or None;
    cu_seqlens int32 [N + 1] on the device, or None with ``num_seqs`` equal
    sequences (default 1).  ``final_state`` may be initial_state.
    """
    T, Hqk, H, dk, dv, N, dev, io = _linear_args(q, k, v, decay, cu_seqlens, num_seqs)
    code = _io_code(io)
    state = (N, H, dv, dk)
    if initial_state is not None:
        _given(initial_state, "initial_state", state, torch.float32, dev)
    if o is not None:
        _given(o, "o", v.shape, io, dev)
    if final_state is not None:
        _given(final_state, "final_state", state, torch.float32, dev)
    need = _linear_bytes(N, T, Hqk, H, dk, dv, code, 0)

    def run(stream_ptr):
        out = torch.empty_like(v) if o is None else o
        fin = final_state
        if fin is None and output_final_state:
            fin = decay.new_empty(state)
        ws, ws_bytes, _keep = _scratch(workspace, need, decay, dev)
        st = load_library().gdr_linear_prefill(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), _at(initial_state),
            _at(cu_seqlens), N, T, Hqk, H, dk, dv, code, out.data_ptr(), _at(fin), ws, ws_bytes,
            stream_ptr)
        _check(st, "gdr_linear_prefill")
        return out, fin

    return _on(dev, stream, run)


def gdr_linear_check_workspace(workspace, stream=None):
    """Raise GdrError(GDR_ERR_DEVICE_TIMEOUT) if a bounded device-side wait of
    the call that used this workspace gave up (synchronises the stream)."""
    _on(workspace.device, stream, lambda stream_ptr: _check(
        load_library().gdr_linear_check_workspace(
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream_ptr),
        "gdr_linear_check_workspace"))


def gdr_linear_decode(q, k, v, decay, state, *, o=None, stream=None):
    """One token per sequence (see include/gdr.h): state is updated in place.

    q, k [N, H_qk, d_k], v [N, H, d_v] (bf16 or fp32); decay [H] fp32; state
    [N, H, d_v, d_k] fp32.  Returns o [N, H, d_v].
    """
    N, Hqk, H, dk, dv, _, dev, io = _linear_args(q, k, v, decay, None, None)
    code = _io_code(io)
    _given(state, "state", (N, H, dv, dk), torch.float32, dev)
    if o is not None:
        _given(o, "o", v.shape, io, dev)

    def run(stream_ptr):
        out = torch.empty_like(v) if o is None else o
        st = load_library().gdr_linear_decode(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), state.data_ptr(), N, Hqk,
            H, dk, dv, code, out.data_ptr(), stream_ptr)
        _check(st, "gdr_linear_decode")
        return out

    return _on(dev, stream, run)


def gdr_linear_backward(q, k, v, decay, initial_state=None, cu_seqlens=None, *, d_o,
                        d_final_state=None, num_seqs=None, want_d_initial_state=True,
                        workspace=None, stream=None):
    """Gradient of <d_o, o> + <d_final_state, final_state> of
    gdr_linear_prefill (see include/gdr.h).

    d_o [T, H, d_v] in the io dtype; d_final_state [N, H, d_v, d_k] fp32 or
    None.  Returns (dq, dk, dv, d_initial_state): the first three in the io
    dtype, the last fp32 (None unless wanted).
    """
    T, Hqk, H, dk, dv, N, dev, io = _linear_args(q, k, v, decay, cu_seqlens, num_seqs)
    code = _io_code(io)
    state = (N, H, dv, dk)
    _given(d_o, "d_o", v.shape, io, dev)
    if initial_state is not None:
        _given(initial_state, "initial_state", state, torch.float32, dev)
    if d_final_state is not None:
        _given(d_final_state, "d_final_state", state, torch.float32, dev)
    need = _linear_bytes(N, T, Hqk, H, dk, dv, code, 1)

    def run(stream_ptr):
        dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dh0 = decay.new_empty(state) if want_d_initial_state else None
        ws, ws_bytes, _keep = _scratch(workspace, need, decay, dev)
        st = load_library().gdr_linear_backward(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), _at(initial_state),
            _at(cu_seqlens), N, T, Hqk, H, dk, dv, code, d_o.data_ptr(), _at(d_final_state),
            dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(), _at(dh0), ws, ws_bytes, stream_ptr)
        _check(st, "gdr_linear_backward")
        return dq, dk_, dv_, dh0

    return _on(dev, stream, run)


def _norm_args(x, weight, gate, residual, next_weight, activation):
    """Checks what the norm's two calls share; returns (rows, dim, device, shape, activation)."""
    _need(x, "x")
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must have at least one dim")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {activation!r}")
    dim, dev, io = _int32(shape[-1], "x's last dimension"), x.device, x.dtype
    if gate is not None:
        _given(gate, "gate", shape, io, dev)
    if residual is not None:
        _given(residual, "residual", shape, io, dev)
    if weight is not None:
        _given(weight, "weight", (dim,), torch.float32, dev)
    if next_weight is not None:
        _given(next_weight, "next_weight", (dim,), torch.float32, dev)
    return x.numel() // dim if dim else 0, dim, dev, shape, act


def gdr_norm_gate(x, weight=None, gate=None, residual=None, next_weight=None, *, scale=1.0,
                  eps=1e-6, activation="silu", y=None, y_norm=None, stream=None):
    """y = residual + scale * act(gate) * norm(x) * weight and y_norm =
    norm(y) * next_weight over the last dimension (see include/gdr.h).

    x, gate, residual [..., dim] (bf16 or fp32); weight, next_weight [dim]
    fp32; everything but x may be None; activation "silu", "sigmoid" or
    "none".  ``y`` may be residual.  Returns (y, y_norm); y_norm is None
    without next_weight.
    """
    rows, dim, dev, shape, act = _norm_args(x, weight, gate, residual, next_weight, activation)
    code = _io_code(x.dtype)
    if y is not None:
        _given(y, "y", shape, x.dtype, dev)
    if y_norm is not None:
        if next_weight is None:
            raise ValueError("y_norm needs next_weight")
        _given(y_norm, "y_norm", shape, x.dtype, dev)

    def run(stream_ptr):
        out = torch.empty_like(x) if y is None else y
        normed = y_norm
        if normed is None and next_weight is not None:
            normed = torch.empty_like(x)
        st = load_library().gdr_norm_gate(
            x.data_ptr(), _at(weight), _at(gate), _at(residual), _at(next_weight), rows, dim,
            float(scale), float(eps), act, code, out.data_ptr(), _at(normed), stream_ptr)
        _check(st, "gdr_norm_gate")
        return out, normed

    return _on(dev, stream, run)


@functools.lru_cache(maxsize=1024)
def _norm_bytes(rows, dim):
    n = ctypes.c_size_t(0)
    _check(load_library().gdr_norm_gate_workspace_size(rows, dim, ctypes.byref(n)),
           "gdr_norm_gate_workspace_size")
    return int(n.value)


def gdr_norm_gate_workspace_size(rows, dim) -> int:
    return _norm_bytes(rows, _int32(dim, "dim"))


def gdr_norm_gate_backward(x, dy=None, dn=None, weight=None, gate=None, residual=None,
                           next_weight=None, *, scale=1.0, eps=1e-6, activation="silu",
                           workspace=None, stream=None):
    """Gradient of <dy, y> + <dn, y_norm> of gdr_norm_gate (see include/gdr.h).

    dy, dn like x, either None.  Returns (dx, dweight, dgate, dresidual,
    dnext_weight): None for an input that was not given, and dnext_weight None
    without dn.
    """
    rows, dim, dev, shape, act = _norm_args(x, weight, gate, residual, next_weight, activation)
    code = _io_code(x.dtype)
    if dy is None and dn is None:
        raise ValueError("dy or dn is required")
    if dy is not None:
        _given(dy, "dy", shape, x.dtype, dev)
    if dn is not None:
        _given(dn, "dn", shape, x.dtype, dev)
        if next_weight is None:
            raise ValueError("dn needs next_weight")
    need = 0 if weight is None and dn is None else _norm_bytes(rows, dim)

    def run(stream_ptr):
        new = lambda like: None if like is None else torch.empty_like(like)  # noqa: E731
        dx, dweight, dgate, dres = new(x), new(weight), new(gate), new(residual)
        dnext = new(next_weight) if dn is not None else None
        ws, ws_bytes, _keep = _scratch(workspace, need, weight if weight is not None else next_weight, dev)
        st = load_library().gdr_norm_gate_backward(
            x.data_ptr(), _at(weight), _at(gate), _at(residual), _at(next_weight), rows, dim,
            float(scale), float(eps), act, code, _at(dy), _at(dn), dx.data_ptr(), _at(dweight),
            _at(dgate), _at(dres), _at(dnext), ws, ws_bytes, stream_ptr)
        _check(st, "gdr_norm_gate_backward")
        return dx, dweight, dgate, dres, dnext

    return _on(dev, stream, run)
