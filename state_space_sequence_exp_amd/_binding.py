"""ctypes binding of libm3ssm (include/m3ssm.h).

Argument marshalling only: every step of the recurrence runs in the HIP
kernels of libm3ssm.so.  PyTorch supplies device memory and the current
stream.  If the library is not built this module raises on first use; there
is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math
import os
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libm3ssm.so")

M3_SUCCESS = 0
M3_ERR_INVALID_VALUE = 1
M3_ERR_NOT_SUPPORTED = 2
M3_ERR_WORKSPACE = 3
M3_ERR_HIP = 4
M3_ERR_CHAIN = 5
M3_F32 = 0
M3_BF16 = 1
M3_CODE_INT8 = 0
M3_CODE_E4M3 = 1
SCAN_CHUNK = 64

# every function declared in include/m3ssm.h
ABI_SYMBOLS = ("m3_version", "m3_status_string", "m3_prefill_workspace_size", "m3_prefill",
               "m3_prefill_workspace_error", "m3_prefill_noalloc", "m3_prefill_from_state", "m3_decode_step", "m3_decode_step_mfma", "m3_block_prepass", "m3_block_postpass",
               "m3_backward_workspace_size", "m3_backward",
               "m3_gated_scan_workspace_size", "m3_gated_scan", "m3_gated_scan_backward",
               "m3_gated_scan_step", "m3_layer_norm", "m3_layer_norm_backward_workspace_size",
               "m3_layer_norm_backward", "m3_state_store", "m3_state_load",
               "m3_decode_step_cached", "m3_causal_conv", "m3_causal_conv_step",
               "m3_selective_scan_workspace_size", "m3_selective_scan", "m3_selective_scan_step",
               "m3_gated_ffn", "m3_gated_ffn_backward_workspace_size", "m3_gated_ffn_backward")


class M3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s" % (where, status_string(status)))


class M3Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim_p", ctypes.c_int64),
                ("dstate_n", ctypes.c_int64), ("rank_r", ctypes.c_int64)]


class M3ScanDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("batch", "seqlen", "channels", "ld_x", "ld_f", "ld_g",
                                              "ld_y", "ld_dx", "ld_df", "ld_dg")]


class M3NormDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("rows", "channels", "ld_x", "ld_residual", "ld_sum",
                                              "ld_y", "ld_dy", "ld_dsum", "ld_dx")]


class M3ConvDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("batch", "seqlen", "channels", "width", "ld_x", "ld_y")]


class M3SelectDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("batch", "seqlen", "channels", "dstate_n", "ld_x", "ld_dt",
                                              "ld_z", "ld_y", "ld_b", "ld_c")]


class M3FfnDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("rows", "channels", "hidden", "ld_x", "ld_wgate", "ld_wup",
                                              "ld_h", "ld_gate", "ld_up", "ld_dh", "ld_dx", "ld_dwgate",
                                              "ld_dwup")]


_lib = None


def load_library(path: Optional[str] = None):
    """Load libm3ssm.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libm3ssm.so not found at %s; build it with "
                           "`python -m state_space_sequence_exp_amd.build`" % p)
    # torch first: it brings its own HIP runtime, and the library must bind
    # to the same one (loaded before torch, the library would start the
    # system runtime, which then sees no device next to torch's)
    import torch  # noqa: F401
    lib = ctypes.CDLL(p)
    vp = ctypes.c_void_p
    dp = ctypes.POINTER(M3Dims)
    lib.m3_version.restype = ctypes.c_int
    lib.m3_version.argtypes = []
    lib.m3_status_string.restype = ctypes.c_char_p
    lib.m3_status_string.argtypes = [ctypes.c_int]
    lib.m3_prefill_workspace_size.restype = ctypes.c_size_t
    lib.m3_prefill_workspace_size.argtypes = [dp, ctypes.c_int, ctypes.c_int]
    lib.m3_prefill.restype = ctypes.c_int
    lib.m3_prefill.argtypes = [dp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp,
                               vp, vp, ctypes.c_size_t, vp]
    lib.m3_prefill_workspace_error.restype = ctypes.c_int
    lib.m3_prefill_workspace_error.argtypes = [vp, ctypes.c_size_t, ctypes.c_int,
                                               ctypes.POINTER(ctypes.c_int), vp]
    lib.m3_prefill_noalloc.restype = ctypes.c_int
    lib.m3_prefill_noalloc.argtypes = [dp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, vp]
    lib.m3_prefill_from_state.restype = ctypes.c_int
    lib.m3_prefill_from_state.argtypes = [dp, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.m3_decode_step.restype = ctypes.c_int
    lib.m3_decode_step.argtypes = [dp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   vp, vp]
    lib.m3_decode_step_mfma.restype = ctypes.c_int
    lib.m3_decode_step_mfma.argtypes = [dp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   vp, vp]
    lib.m3_backward_workspace_size.restype = ctypes.c_size_t
    lib.m3_backward_workspace_size.argtypes = [dp, ctypes.c_int]
    lib.m3_backward.restype = ctypes.c_int
    lib.m3_backward.argtypes = [dp, ctypes.c_int] + [vp] * 17 + [ctypes.c_size_t, vp]
    lib.m3_block_prepass.restype = ctypes.c_int
    lib.m3_block_prepass.argtypes = [dp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp,
                                     ctypes.c_float, vp, vp, vp, vp]
    lib.m3_block_postpass.restype = ctypes.c_int
    lib.m3_block_postpass.argtypes = [dp, ctypes.c_int, vp, vp, vp, vp]
    sp, np_ = ctypes.POINTER(M3ScanDims), ctypes.POINTER(M3NormDims)
    i, sz, i64 = ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
    lib.m3_gated_scan_workspace_size.restype = sz
    lib.m3_gated_scan_workspace_size.argtypes = [sp, i]
    lib.m3_gated_scan.restype = i
    lib.m3_gated_scan.argtypes = [sp, i] + [vp] * 8 + [sz, vp]
    lib.m3_gated_scan_backward.restype = i
    lib.m3_gated_scan_backward.argtypes = [sp, i] + [vp] * 11 + [sz, vp]
    lib.m3_gated_scan_step.restype = i
    lib.m3_gated_scan_step.argtypes = [sp, i] + [vp] * 7
    lib.m3_layer_norm.restype = i
    lib.m3_layer_norm.argtypes = [np_, i] + [vp] * 4 + [ctypes.c_float] + [vp] * 5
    lib.m3_layer_norm_backward_workspace_size.restype = sz
    lib.m3_layer_norm_backward_workspace_size.argtypes = [np_, i]
    lib.m3_layer_norm_backward.restype = i
    lib.m3_layer_norm_backward.argtypes = [np_, i] + [vp] * 10 + [sz, vp]
    lib.m3_state_store.restype = i
    lib.m3_state_store.argtypes = [dp, i, vp, vp, vp, vp, i64, vp]
    lib.m3_state_load.restype = i
    lib.m3_state_load.argtypes = [dp, i, i, vp, vp, vp, i64, vp, vp]
    lib.m3_decode_step_cached.restype = i
    lib.m3_decode_step_cached.argtypes = [dp, i, i, vp, vp, vp, i64] + [vp] * 11
    cp, ep, fp = (ctypes.POINTER(t) for t in (M3ConvDims, M3SelectDims, M3FfnDims))
    lib.m3_causal_conv.restype = i
    lib.m3_causal_conv.argtypes = [cp, i, vp, vp, vp, i] + [vp] * 5
    lib.m3_causal_conv_step.restype = i
    lib.m3_causal_conv_step.argtypes = [cp, i, vp, vp, i64, vp, vp, vp, i, vp, vp]
    lib.m3_selective_scan_workspace_size.restype = sz
    lib.m3_selective_scan_workspace_size.argtypes = [ep, i]
    lib.m3_selective_scan.restype = i
    lib.m3_selective_scan.argtypes = [ep, i] + [vp] * 8 + [i] + [vp] * 5 + [sz, vp]
    lib.m3_selective_scan_step.restype = i
    lib.m3_selective_scan_step.argtypes = [ep, i, vp, vp, i64] + [vp] * 8 + [i, vp, vp]
    lib.m3_gated_ffn.restype = i
    lib.m3_gated_ffn.argtypes = [fp, i] + [vp] * 7
    lib.m3_gated_ffn_backward_workspace_size.restype = sz
    lib.m3_gated_ffn_backward_workspace_size.argtypes = [fp, i]
    lib.m3_gated_ffn_backward.restype = i
    lib.m3_gated_ffn_backward.argtypes = [fp, i] + [vp] * 10 + [sz, vp]
    if path is None:
        _lib = lib
    return lib


def version() -> int:
    return load_library().m3_version()


def status_string(status: int) -> str:
    return load_library().m3_status_string(int(status)).decode()


def _dims(batch, seqlen, nheads, P, N, R) -> M3Dims:
    return M3Dims(int(batch), int(seqlen), int(nheads), int(P), int(N), int(R))


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return M3_F32
    if t.dtype == torch.bfloat16:
        return M3_BF16
    raise TypeError("x, B, C must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s: on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def prefill_workspace_size(batch, seqlen, nheads, P, N, R, chunk, dtype) -> int:
    """Bytes of workspace m3_prefill needs (0: nothing to do, or unsupported)."""
    import torch
    code = dtype if isinstance(dtype, int) else (M3_BF16 if dtype == torch.bfloat16 else M3_F32)
    d = _dims(batch, seqlen, nheads, P, N, R)
    return int(load_library().m3_prefill_workspace_size(ctypes.byref(d), int(chunk), code))


def prefill_workspace_error(workspace, *, clear: bool = False, stream=None) -> int:
    """The error word of a prefill workspace once the stream's work has
    finished (m3_prefill_workspace_error; synchronises the stream): 0 when
    every chain wait completed, 1 after a timed-out wait (outputs NaN), 2
    after dirty counters.  With clear=True a nonzero word is reset."""
    word = ctypes.c_int(0)
    nbytes = workspace.numel() * workspace.element_size()
    st = load_library().m3_prefill_workspace_error(_ptr(workspace), nbytes, int(bool(clear)),
                                                   ctypes.byref(word), _stream(stream))
    if st not in (M3_SUCCESS, M3_ERR_CHAIN):
        raise M3Error(st, "m3_prefill_workspace_error")
    return int(word.value)


def prefill(x, dt, A, lam, theta, B, C, chunk: int, *, h0=None, x_prev=None, B_prev=None,
            y=None, h_final=None, want_h_final: bool = True, workspace=None,
            check: bool = False, stream=None) -> Tuple:
    """Chunked prefill on the GPU.

    x [Bt,T,H,R,P] (or [Bt,T,H,P] for R=1); B, C [Bt,T,H,R,N] (or [Bt,T,H,N]);
    dt, lam [Bt,T,H]; theta [Bt,T,H,N/2]; A [H].  x, B, C float32 or
    bfloat16 (same dtype), the rest float32, all contiguous on one GPU.
    lam=None gives the exponential-Euler rule (lam = 1, Mamba-2's
    discretisation) and theta=None a real state (no rotation).
    To continue a sequence pass h0 [Bt,H,N,P] float32 (the state before the
    first token) and/or x_prev [Bt,H,R,P] with B_prev [Bt,H,R,N] (the
    previous token's x and B, x's dtype; R axis optional for R=1); this calls
    m3_prefill_from_state.  h_final may be h0 (in-place update).
    check=True synchronises the stream after the call and raises M3Error
    (M3_ERR_CHAIN) if the workspace's error word is set.
    Returns (y with x's shape and dtype, h_final [Bt,H,N,P] float32 or None).
    """
    import torch
    lib = load_library()
    squeeze = x.dim() == 4
    x5 = x.unsqueeze(3) if squeeze else x
    B5 = B.unsqueeze(3) if B.dim() == 4 else B
    C5 = C.unsqueeze(3) if C.dim() == 4 else C
    nb, nt, nh, nr, npd = x5.shape
    nn = B5.shape[-1]
    dev = x.device
    code = _dtype_code(x)
    _check(x5, "x", x.dtype, (nb, nt, nh, nr, npd), dev)
    _check(B5, "B", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(C5, "C", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(dt, "dt", torch.float32, (nb, nt, nh), dev)
    if lam is not None:
        _check(lam, "lam", torch.float32, (nb, nt, nh), dev)
    if theta is not None:
        _check(theta, "theta", torch.float32, (nb, nt, nh, nn // 2), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check(y, "y", x.dtype, tuple(x.shape), dev)
    if h_final is None and want_h_final:
        h_final = torch.empty((nb, nh, nn, npd), dtype=torch.float32, device=dev)
    elif h_final is not None:
        _check(h_final, "h_final", torch.float32, (nb, nh, nn, npd), dev)
    cont = h0 is not None or x_prev is not None or B_prev is not None
    if h0 is not None:
        _check(h0, "h0", torch.float32, (nb, nh, nn, npd), dev)
    if (x_prev is None) != (B_prev is None):
        raise ValueError("x_prev and B_prev go together")
    if x_prev is not None:
        x_prev = x_prev.unsqueeze(2) if x_prev.dim() == 3 else x_prev
        B_prev = B_prev.unsqueeze(2) if B_prev.dim() == 3 else B_prev
        _check(x_prev, "x_prev", x.dtype, (nb, nh, nr, npd), dev)
        _check(B_prev, "B_prev", x.dtype, (nb, nh, nr, nn), dev)
    d = _dims(nb, nt, nh, npd, nn, nr)
    need = int(lib.m3_prefill_workspace_size(ctypes.byref(d), int(chunk), code))
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if cont:
        st = lib.m3_prefill_from_state(ctypes.byref(d), code, int(chunk), _ptr(h0), _ptr(x_prev),
                                       _ptr(B_prev), _ptr(x5), _ptr(dt), _ptr(A), _ptr(lam),
                                       _ptr(theta), _ptr(B5), _ptr(C5), _ptr(y), _ptr(h_final),
                                       _ptr(workspace), ws_bytes, _stream(stream))
    else:
        st = lib.m3_prefill(ctypes.byref(d), code, int(chunk), _ptr(x5), _ptr(dt), _ptr(A),
                            _ptr(lam), _ptr(theta), _ptr(B5), _ptr(C5), _ptr(y), _ptr(h_final),
                            _ptr(workspace), ws_bytes, _stream(stream))
    if st != M3_SUCCESS:
        raise M3Error(st, "m3_prefill_from_state" if cont else "m3_prefill")
    if check and workspace is not None:
        if prefill_workspace_error(workspace, stream=stream) != 0:
            raise M3Error(M3_ERR_CHAIN, "m3_prefill_from_state" if cont else "m3_prefill")
    return y, h_final


# device scratch of m3_prefill_noalloc, per GPU (M3_PREFILL_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 32 << 20


def prefill_noalloc(x, dt, A, lam, theta, B, C, chunk: int, y, h_final=None,
                    stream=None) -> Tuple:
    """Chunked prefill through m3_prefill_noalloc: no workspace, and nothing
    allocated by this call (y, and h_final if wanted, are the caller's).  The
    library's per-GPU scratch stands in for the workspace, so calls that
    overlap on one GPU race.  Shapes as for prefill()."""
    import torch
    lib = load_library()
    x5 = x.unsqueeze(3) if x.dim() == 4 else x
    B5 = B.unsqueeze(3) if B.dim() == 4 else B
    C5 = C.unsqueeze(3) if C.dim() == 4 else C
    nb, nt, nh, nr, npd = x5.shape
    nn = B5.shape[-1]
    dev = x.device
    code = _dtype_code(x)
    _check(x5, "x", x.dtype, (nb, nt, nh, nr, npd), dev)
    _check(B5, "B", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(C5, "C", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(dt, "dt", torch.float32, (nb, nt, nh), dev)
    if lam is not None:
        _check(lam, "lam", torch.float32, (nb, nt, nh), dev)
    if theta is not None:
        _check(theta, "theta", torch.float32, (nb, nt, nh, nn // 2), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    _check(y, "y", x.dtype, tuple(x.shape), dev)
    if h_final is not None:
        _check(h_final, "h_final", torch.float32, (nb, nh, nn, npd), dev)
    d = _dims(nb, nt, nh, npd, nn, nr)
    st = lib.m3_prefill_noalloc(ctypes.byref(d), code, int(chunk), _ptr(x5), _ptr(dt), _ptr(A),
                                _ptr(lam), _ptr(theta), _ptr(B5), _ptr(C5), _ptr(y),
                                _ptr(h_final), _stream(stream))
    if st != M3_SUCCESS:
        raise M3Error(st, "m3_prefill_noalloc")
    return y, h_final


def decode_step(h, x_t, x_prev, B_t, B_prev, C_t, dt, A, lam, theta, *, h_out=None, y=None,
                stream=None, matrix_cores: bool = False) -> Tuple:
    """One decode step on the GPU.

    h [S,H,N,P] float32; x_t, x_prev [S,H,R,P]; B_t, B_prev, C_t [S,H,R,N]
    (float32 or bfloat16); dt, lam [S,H]; theta [S,H,N/2]; A [H].
    lam=None gives the exponential-Euler rule (lam = 1; x_prev and B_prev
    are then not read and may be None) and theta=None a real state.
    h_out defaults to h itself (in-place update).  Returns (y_t [S,H,R,P],
    h_out).  matrix_cores=True calls m3_decode_step_mfma (the rank-2R
    update on MFMA; R 2 or 4, P 64, N a multiple of 16 up to 128).
    """
    import torch
    lib = load_library()
    ns, nh, nn, npd = h.shape
    nr = x_t.shape[2]
    dev = h.device
    code = _dtype_code(x_t)
    _check(h, "h", torch.float32, (ns, nh, nn, npd), dev)
    if lam is None and x_prev is None and B_prev is None:
        x_prev = B_prev = None
    elif x_prev is None or B_prev is None:
        raise ValueError("x_prev and B_prev are required with lam")
    for name, t in (("x_t", x_t), ("x_prev", x_prev)):
        if t is not None:
            _check(t, name, x_t.dtype, (ns, nh, nr, npd), dev)
    for name, t in (("B_t", B_t), ("B_prev", B_prev), ("C_t", C_t)):
        if t is not None:
            _check(t, name, x_t.dtype, (ns, nh, nr, nn), dev)
    _check(dt, "dt", torch.float32, (ns, nh), dev)
    if lam is not None:
        _check(lam, "lam", torch.float32, (ns, nh), dev)
    if theta is not None:
        _check(theta, "theta", torch.float32, (ns, nh, nn // 2), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    if h_out is None:
        h_out = h
    else:
        _check(h_out, "h_out", torch.float32, (ns, nh, nn, npd), dev)
    if y is None:
        y = torch.empty((ns, nh, nr, npd), dtype=x_t.dtype, device=dev)
    else:
        _check(y, "y", x_t.dtype, (ns, nh, nr, npd), dev)
    d = _dims(ns, 1, nh, npd, nn, nr)
    fn = lib.m3_decode_step_mfma if matrix_cores else lib.m3_decode_step
    st = fn(ctypes.byref(d), code, _ptr(h), _ptr(h_out), _ptr(x_t), _ptr(x_prev), _ptr(B_t),
            _ptr(B_prev), _ptr(C_t), _ptr(dt), _ptr(A), _ptr(lam), _ptr(theta), _ptr(y),
            _stream(stream))
    if st != M3_SUCCESS:
        raise M3Error(st, "m3_decode_step_mfma" if matrix_cores else "m3_decode_step")
    return y, h_out


def block_prepass(x, B, C, norm_B, norm_C, bias_B, bias_C, up, eps: float = 1e-6, *,
                  x_out=None, B_out=None, C_out=None, stream=None) -> Tuple:
    """BCNorm + bias on B and C, MIMO up-projection of x (m3_block_prepass).

    x [Bt,T,H,P]; B, C [Bt,T,H,R,N] (float32 or bfloat16, same dtype);
    norm_B, norm_C [H,N]; bias_B, bias_C [H,R,N]; up [H,R,P] float32.
    Returns (X [Bt,T,H,R,P], B~, C~ [Bt,T,H,R,N]) in x's dtype.
    """
    import torch
    lib = load_library()
    nb, nt, nh, npd = x.shape
    nr, nn = B.shape[3], B.shape[4]
    dev = x.device
    code = _dtype_code(x)
    _check(x, "x", x.dtype, (nb, nt, nh, npd), dev)
    _check(B, "B", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(C, "C", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(norm_B, "norm_B", torch.float32, (nh, nn), dev)
    _check(norm_C, "norm_C", torch.float32, (nh, nn), dev)
    _check(bias_B, "bias_B", torch.float32, (nh, nr, nn), dev)
    _check(bias_C, "bias_C", torch.float32, (nh, nr, nn), dev)
    _check(up, "up", torch.float32, (nh, nr, npd), dev)
    if x_out is None:
        x_out = torch.empty((nb, nt, nh, nr, npd), dtype=x.dtype, device=dev)
    if B_out is None:
        B_out = torch.empty_like(B)
    if C_out is None:
        C_out = torch.empty_like(C)
    _check(x_out, "x_out", x.dtype, (nb, nt, nh, nr, npd), dev)
    _check(B_out, "B_out", x.dtype, tuple(B.shape), dev)
    _check(C_out, "C_out", x.dtype, tuple(C.shape), dev)
    d = _dims(nb, nt, nh, npd, nn, nr)
    st = lib.m3_block_prepass(ctypes.byref(d), code, _ptr(x), _ptr(B), _ptr(C), _ptr(norm_B),
                              _ptr(norm_C), _ptr(bias_B), _ptr(bias_C), _ptr(up),
                              ctypes.c_float(eps), _ptr(x_out), _ptr(B_out), _ptr(C_out),
                              _stream(stream))
    if st != M3_SUCCESS:
        raise M3Error(st, "m3_block_prepass")
    return x_out, B_out, C_out


def block_postpass(y, down, *, y_out=None, stream=None):
    """MIMO down-projection y_out = sum_r down[h,r] * y[r] (m3_block_postpass).

    y [Bt,T,H,R,P] float32 or bfloat16; down [H,R,P] float32.
    Returns y_out [Bt,T,H,P] in y's dtype.
    """
    import torch
    lib = load_library()
    nb, nt, nh, nr, npd = y.shape
    dev = y.device
    code = _dtype_code(y)
    _check(y, "y", y.dtype, (nb, nt, nh, nr, npd), dev)
    _check(down, "down", torch.float32, (nh, nr, npd), dev)
    if y_out is None:
        y_out = torch.empty((nb, nt, nh, npd), dtype=y.dtype, device=dev)
    _check(y_out, "y_out", y.dtype, (nb, nt, nh, npd), dev)
    # the state size does not enter the post-pass; any supported value
    d = _dims(nb, nt, nh, npd, 64, nr)
    st = lib.m3_block_postpass(ctypes.byref(d), code, _ptr(y), _ptr(down), _ptr(y_out),
                               _stream(stream))
    if st != M3_SUCCESS:
        raise M3Error(st, "m3_block_postpass")
    return y_out


def backward_workspace_size(batch, seqlen, nheads, P, N, R, dtype) -> int:
    """Bytes of workspace m3_backward needs (0: nothing to do, or unsupported)."""
    import torch
    code = dtype if isinstance(dtype, int) else (M3_BF16 if dtype == torch.bfloat16 else M3_F32)
    d = _dims(batch, seqlen, nheads, P, N, R)
    return int(load_library().m3_backward_workspace_size(ctypes.byref(d), code))


def backward(x, dt, A, lam, theta, B, C, dy, *, dh_final=None, workspace=None, stream=None):
    """Gradients of sum(y * dy) (+ sum(h_final * dh_final)) for the prefill
    inputs (m3_backward).  Shapes as for prefill; dy has x's shape and dtype.
    Returns a dict of float32 gradients: x, dt, A, lam, theta, B, C."""
    import torch
    lib = load_library()
    squeeze = x.dim() == 4
    x5 = x.unsqueeze(3) if squeeze else x
    B5 = B.unsqueeze(3) if B.dim() == 4 else B
    C5 = C.unsqueeze(3) if C.dim() == 4 else C
    dy5 = dy.unsqueeze(3) if dy.dim() == 4 else dy
    nb, nt, nh, nr, npd = x5.shape
    nn = B5.shape[-1]
    dev = x.device
    code = _dtype_code(x)
    _check(x5, "x", x.dtype, (nb, nt, nh, nr, npd), dev)
    _check(dy5, "dy", x.dtype, (nb, nt, nh, nr, npd), dev)
    _check(B5, "B", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(C5, "C", x.dtype, (nb, nt, nh, nr, nn), dev)
    _check(dt, "dt", torch.float32, (nb, nt, nh), dev)
    _check(lam, "lam", torch.float32, (nb, nt, nh), dev)
    _check(theta, "theta", torch.float32, (nb, nt, nh, nn // 2), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    if dh_final is not None:
        _check(dh_final, "dh_final", torch.float32, (nb, nh, nn, npd), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"x": torch.empty((nb, nt, nh, nr, npd), **f32), "dt": torch.empty((nb, nt, nh), **f32),
         "A": torch.empty((nh,), **f32), "lam": torch.empty((nb, nt, nh), **f32),
         "theta": torch.empty((nb, nt, nh, nn // 2), **f32),
         "B": torch.empty((nb, nt, nh, nr, nn), **f32), "C": torch.empty((nb, nt, nh, nr, nn), **f32)}
    d = _dims(nb, nt, nh, npd, nn, nr)
    need = int(lib.m3_backward_workspace_size(ctypes.byref(d), code))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.m3_backward(ctypes.byref(d), code, _ptr(x5), _ptr(dt), _ptr(A), _ptr(lam),
                         _ptr(theta), _ptr(B5), _ptr(C5), _ptr(dy5), _ptr(dh_final),
                         _ptr(g["x"]), _ptr(g["dt"]), _ptr(g["A"]), _ptr(g["lam"]),
                         _ptr(g["theta"]), _ptr(g["B"]), _ptr(g["C"]), _ptr(workspace),
                         ws_bytes, _stream(stream))
    if st != M3_SUCCESS:
        raise M3Error(st, "m3_backward")
    if squeeze:
        g["x"] = g["x"].squeeze(3)
    return g


# ---- operators beside the recurrence ------------------------------------------
# A call's device is its first tensor's.  Where that is not the current device
# the call is made with it current, on that device's current stream.
#
# Several of these run for a few microseconds, less than a careless wrapper
# takes, so the checks of a call ask each tensor for as little as they can.

_types = None


def _type_code(dtype) -> int:
    """M3_F32 or M3_BF16 of a torch type (or of the code itself)."""
    global _types
    if _types is None:
        import torch
        _types = {torch.float32: M3_F32, torch.bfloat16: M3_BF16, M3_F32: M3_F32, M3_BF16: M3_BF16}
    code = _types.get(dtype)
    if code is None:
        raise TypeError("expected float32 or bfloat16, got %s" % dtype)
    return code


def _launch(dev: int, fn, *args):
    """fn(*args, stream) with device `dev` and its current stream; raises M3Error."""
    import torch
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != M3_SUCCESS:
        raise M3Error(st, fn.__name__)


def _streamed(fn):
    """A function that works on the current stream, with an argument `stream`
    (a torch stream or its handle, of the first tensor's device) that makes
    another one current for the call: what the call allocates and zero-fills
    is then ordered with its kernels."""
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None or not (args or first in kw):
            return fn(*args, **kw)
        import torch
        dev = (args[0] if args else kw[first]).get_device()
        _gpu(dev)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=dev)
        if stream.device.index != dev:
            raise ValueError("stream: of %s, expected the first tensor's device" % stream.device)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _at(t):
    return None if t is None else t.data_ptr()


def _same(t, name, dtype, shape, dev: int):
    """A dense array of this type and shape on device `dev`."""
    if t.dtype is not dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s: on %s, expected the first tensor's device" % (name, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name, dtype, shape, dev: int) -> int:
    """Checks an array of rows [..., D] whose channels are contiguous and whose
    rows follow each other at one distance (a dense array, or a slice of wider
    rows); returns that distance in elements."""
    if t.dtype is not dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s: on %s, expected the first tensor's device" % (name, t.device))
    if t.is_contiguous():
        return 0
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s: its last dimension must be contiguous" % name)
    ld = step = None
    for n, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = step = st
        if st != step or st < shape[-1]:
            raise ValueError("%s: its rows must follow each other at one distance" % name)
        step *= n
    return 0 if ld is None else ld


def _gpu(dev: int):
    if dev < 0:
        raise ValueError("tensors must be on a GPU")


def _like(x, dense: bool):
    """A new dense array of x's shape and type."""
    import torch
    return torch.empty_like(x) if dense else x.new_empty(x.shape)


def _code_of(codes) -> int:
    import torch
    if codes.dtype == torch.int8:
        return M3_CODE_INT8
    if codes.dtype == torch.float8_e4m3fn:
        return M3_CODE_E4M3
    raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)


def gated_scan_workspace_size(batch, seqlen, channels, dtype) -> int:
    """Bytes of workspace gated_scan and gated_scan_backward need (0: none)."""
    d = M3ScanDims(int(batch), int(seqlen), int(channels))
    return int(load_library().m3_gated_scan_workspace_size(ctypes.byref(d), _type_code(dtype)))


def _scan_workspace(lib, d, code, workspace, dev):
    import torch
    need = int(lib.m3_gated_scan_workspace_size(ctypes.byref(d), code))
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the first tensor's device")
    return workspace, workspace.nbytes


@_streamed
def gated_scan(x, f, g=None, *, h0=None, y=None, h_last=None, want_states: bool = False,
               states=None, workspace=None) -> Tuple:
    """Gated linear recurrence over a sequence (m3_gated_scan):
    h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(f), y = h * silu(g)
    (y = h without g).

    x, f, g [B,T,D] float32 or bfloat16 (one type), channels contiguous and
    tokens at one distance (a slice of a wider projection is read in place).
    h0 [B,D] float32 or None (zeros).  f = +inf passes the state on without
    looking at x (padding), f = -inf starts afresh (a packed document).
    want_states keeps the state entering every 64 tokens, for the backward.
    A workspace (gated_scan_workspace_size bytes, zero-filled once) may be
    kept for later calls; calls that overlap need distinct ones.  Without one
    every call allocates and zero-fills its own (about 5 us a call).
    y, h_last and states may be given; they must not overlap an input or
    each other.
    Returns (y, h_last [B,D] float32, states [B,ceil(T/64),D] float32 or None).
    """
    import torch
    lib = _lib or load_library()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if len(shape) != 3:
        raise ValueError("x: expected [B, T, D], got %s" % (tuple(shape),))
    nb, nt, nd = shape
    code = _type_code(dt)
    ld = _rows(x, "x", dt, shape, dev)
    d = M3ScanDims(nb, nt, nd, ld, _rows(f, "f", dt, shape, dev),
                   0 if g is None else _rows(g, "g", dt, shape, dev))
    nc = -(-nt // SCAN_CHUNK)
    if h0 is not None:
        _same(h0, "h0", torch.float32, (nb, nd), dev)
    if h_last is not None:
        _same(h_last, "h_last", torch.float32, (nb, nd), dev)
    if states is not None:
        _same(states, "states", torch.float32, (nb, nc, nd), dev)
    if y is not None:
        d.ld_y = _rows(y, "y", dt, shape, dev)
    _gpu(dev)
    if y is None:
        y = _like(x, ld == 0)
    if h_last is None:
        h_last = x.new_empty((nb, nd), dtype=torch.float32)
    if states is None and want_states:
        states = x.new_empty((nb, nc, nd), dtype=torch.float32)
    workspace, ws_bytes = _scan_workspace(lib, d, code, workspace, dev)
    _launch(dev, lib.m3_gated_scan, ctypes.byref(d), code, _at(x), _at(f), _at(g),
            _at(h0), _at(y), _at(h_last), _at(states), _at(workspace), ws_bytes)
    return y, h_last, states


@_streamed
def gated_scan_backward(dy, x, f, g, states, *, dh_last=None, dx=None, df=None, dg=None,
                        workspace=None):
    """Gradients of sum(y * dy) (+ sum(h_last * dh_last)) for gated_scan's
    inputs (m3_gated_scan_backward).  `states` is what gated_scan kept for the
    same inputs; g None when it had none.  dx, df, dg may be given (slices of
    a wider gradient).  Returns a dict: x, f, g (absent without g) in the
    inputs' type, h0 [B,D] float32."""
    import torch
    lib = _lib or load_library()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if len(shape) != 3:
        raise ValueError("x: expected [B, T, D], got %s" % (tuple(shape),))
    nb, nt, nd = shape
    code = _type_code(dt)
    _same(states, "states", torch.float32, (nb, -(-nt // SCAN_CHUNK), nd), dev)
    if dh_last is not None:
        _same(dh_last, "dh_last", torch.float32, (nb, nd), dev)
    if g is None and dg is not None:
        raise ValueError("dg without g")
    rows = lambda t, name: 0 if t is None else _rows(t, name, dt, shape, dev)
    d = M3ScanDims(nb, nt, nd, rows(x, "x"), rows(f, "f"), rows(g, "g"),
                   _rows(dy, "dy", dt, shape, dev), rows(dx, "dx"), rows(df, "df"), rows(dg, "dg"))
    _gpu(dev)
    new = lambda t: _like(x, d.ld_x == 0) if t is None else t
    dx, df, dg = new(dx), new(df), None if g is None else new(dg)
    dh0 = states.new_empty((nb, nd))
    workspace, ws_bytes = _scan_workspace(lib, d, code, workspace, dev)
    _launch(dev, lib.m3_gated_scan_backward, ctypes.byref(d), code, _at(dy), _at(x),
            _at(f), _at(g), _at(states), _at(dh_last), _at(dx), _at(df), _at(dg),
            _at(dh0), _at(workspace), ws_bytes)
    out = {"x": dx, "f": df, "h0": dh0}
    if g is not None:
        out["g"] = dg
    return out


@_streamed
def gated_scan_step(h, x, f, g=None, *, h_out=None, y=None) -> Tuple:
    """One token of the gated linear recurrence (m3_gated_scan_step).

    h [B,D] float32; x, f, g [B,D] float32 or bfloat16.  h_out defaults to h
    itself (in-place update); y must not lie over either.  Returns (y [B,D],
    h_out)."""
    import torch
    lib = _lib or load_library()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if len(shape) != 2:
        raise ValueError("x: expected [B, D], got %s" % (tuple(shape),))
    code = _type_code(dt)
    ld = _rows(x, "x", dt, shape, dev)
    d = M3ScanDims(shape[0], 1, shape[1], ld, _rows(f, "f", dt, shape, dev),
                   0 if g is None else _rows(g, "g", dt, shape, dev))
    _same(h, "h", torch.float32, shape, dev)
    if h_out is None:
        h_out = h
    else:
        _same(h_out, "h_out", torch.float32, shape, dev)
    if y is not None:
        d.ld_y = _rows(y, "y", dt, shape, dev)
    _gpu(dev)
    if y is None:
        y = _like(x, ld == 0)
    _launch(dev, lib.m3_gated_scan_step, ctypes.byref(d), code, _at(h), _at(h_out),
            _at(x), _at(f), _at(g), _at(y))
    return y, h_out


@_streamed
def layer_norm(x, weight, bias=None, eps: float = 1e-5, *, residual=None, y=None, sum_out=None,
               want_stats: bool = True) -> Tuple:
    """Layer norm over the last dimension with the residual sum fused
    (m3_layer_norm): s = x + residual, y = (s - mean) rstd weight + bias.

    x, residual [..., D] float32 or bfloat16, D <= 16384, rows at one
    distance; weight, bias [D] float32.  sum_out may be x or residual (in
    place).  Returns (y, s, mean, rstd): s is x itself without a residual
    (None where y took its place), mean and rstd [...] float32 (None without
    want_stats)."""
    import torch
    lib = _lib or load_library()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if len(shape) < 1:
        raise ValueError("x: expected [..., D]")
    code = _type_code(dt)
    nd = shape[-1]
    rows = math.prod(shape[:-1])
    ld = _rows(x, "x", dt, shape, dev)
    d = M3NormDims(rows, nd, ld)
    _same(weight, "weight", torch.float32, (nd,), dev)
    if bias is not None:
        _same(bias, "bias", torch.float32, (nd,), dev)
    if residual is not None:
        d.ld_residual = _rows(residual, "residual", dt, shape, dev)
    if sum_out is not None:
        d.ld_sum = _rows(sum_out, "sum_out", dt, shape, dev)
    if y is not None:
        d.ld_y = _rows(y, "y", dt, shape, dev)
    _gpu(dev)
    if residual is not None and sum_out is None:
        sum_out = _like(x, ld == 0)
    s = x if sum_out is None else sum_out
    if y is None:
        y = _like(x, ld == 0)
    elif s is x and y.data_ptr() == x.data_ptr():
        s = None
    mean = rstd = None
    if want_stats:
        mean = weight.new_empty(shape[:-1])
        rstd = torch.empty_like(mean)
    _launch(dev, lib.m3_layer_norm, ctypes.byref(d), code, _at(x), _at(residual),
            _at(weight), _at(bias), float(eps), _at(y), _at(sum_out), _at(mean), _at(rstd))
    return y, s, mean, rstd


@_streamed
def layer_norm_backward(dy, s, weight, mean, rstd, *, dsum=None, dx=None, want_bias: bool = True,
                        workspace=None):
    """Gradients of layer_norm (m3_layer_norm_backward): s, mean and rstd as
    layer_norm returned them, dsum the gradient that reaches s past the norm
    (the residual stream's).  dx may be dy or dsum (in place).  Returns a
    dict: x (the gradient of x and of residual) in s's type, weight and bias
    [D] float32 (bias absent without want_bias)."""
    import torch
    lib = _lib or load_library()
    shape, dev, dt = s.shape, s.get_device(), s.dtype
    if len(shape) < 1:
        raise ValueError("s: expected [..., D]")
    code = _type_code(dt)
    nd = shape[-1]
    d = M3NormDims(math.prod(shape[:-1]), nd)
    d.ld_sum = _rows(s, "s", dt, shape, dev)
    d.ld_dy = _rows(dy, "dy", dt, shape, dev)
    _same(weight, "weight", torch.float32, (nd,), dev)
    _same(mean, "mean", torch.float32, shape[:-1], dev)
    _same(rstd, "rstd", torch.float32, shape[:-1], dev)
    if dsum is not None:
        d.ld_dsum = _rows(dsum, "dsum", dt, shape, dev)
    if dx is not None:
        d.ld_dx = _rows(dx, "dx", dt, shape, dev)
    _gpu(dev)
    if dx is None:
        dx = _like(s, d.ld_sum == 0)
    dw = torch.empty_like(weight)
    db = torch.empty_like(weight) if want_bias else None
    need = int(lib.m3_layer_norm_backward_workspace_size(ctypes.byref(d), code))
    if workspace is None and need > 0:
        workspace = weight.new_empty((need + 3) // 4)
    elif workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the first tensor's device")
    ws_bytes = 0 if workspace is None else workspace.nbytes
    _launch(dev, lib.m3_layer_norm_backward, ctypes.byref(d), code, _at(dy), _at(s),
            _at(weight), _at(mean), _at(rstd), _at(dsum), _at(dx), _at(dw),
            _at(db), _at(workspace), ws_bytes)
    out = {"x": dx, "weight": dw}
    if want_bias:
        out["bias"] = db
    return out


def state_cache(n_slots, nheads, N, P, dtype=None, device="cuda") -> Tuple:
    """An empty 8-bit state cache: codes [n_slots,H,N,P] (int8, or
    float8_e4m3fn by dtype) and scales [n_slots,H,N] float32, all zero states."""
    import torch
    if dtype not in (None, torch.int8, torch.float8_e4m3fn):
        raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % dtype)
    codes = torch.zeros((n_slots, nheads, N, P), dtype=torch.int8, device=device)
    scales = torch.zeros((n_slots, nheads, N), dtype=torch.float32, device=device)
    return codes.view(dtype or torch.int8), scales


def _cache_same(codes, scales, slots, dev):
    import torch
    if codes.dim() != 4:
        raise ValueError("codes: expected [slots, H, N, P], got %s" % (tuple(codes.shape),))
    code = _code_of(codes)
    _same(codes, "codes", codes.dtype, codes.shape, dev)
    _same(scales, "scales", torch.float32, codes.shape[:3], dev)
    if slots is not None:
        if slots.dim() != 1:
            raise ValueError("slots: expected [batch], got %s" % (tuple(slots.shape),))
        _same(slots, "slots", torch.int32, slots.shape, dev)
    return code


@_streamed
def state_store(h, codes, scales, slots=None) -> None:
    """Quantises states h [S,H,N,P] float32 into the cache's slots
    (m3_state_store).  slots [S] int32, negative or past the pool: idle; None:
    state i into slot i."""
    import torch
    lib = _lib or load_library()
    dev = codes.get_device()
    code = _cache_same(codes, scales, slots, dev)
    ns = h.shape[0] if slots is None else slots.shape[0]
    _same(h, "h", torch.float32, (ns,) + codes.shape[1:], dev)
    _gpu(dev)
    n, nh, nn, npd = codes.shape
    d = M3Dims(ns, 1, nh, npd, nn, 1)
    _launch(dev, lib.m3_state_store, ctypes.byref(d), code, _at(h), _at(codes),
            _at(scales), _at(slots), n)


@_streamed
def state_load(codes, scales, slots=None, *, dtype=None, h=None):
    """The states of the cache's slots [S,H,N,P] as float32 (or bfloat16 by
    dtype) (m3_state_load); zeros for idle slots; slots None: the whole pool."""
    import torch
    lib = _lib or load_library()
    dev = codes.get_device()
    code = _cache_same(codes, scales, slots, dev)
    n, nh, nn, npd = codes.shape
    ns = n if slots is None else slots.shape[0]
    if h is not None:
        _same(h, "h", dtype or h.dtype, (ns, nh, nn, npd), dev)
    elif dtype not in (None, torch.float32, torch.bfloat16):
        raise TypeError("expected float32 or bfloat16, got %s" % dtype)
    _gpu(dev)
    if h is None:
        h = scales.new_empty((ns, nh, nn, npd), dtype=dtype or torch.float32)
    d = M3Dims(ns, 1, nh, npd, nn, 1)
    _launch(dev, lib.m3_state_load, ctypes.byref(d), code, _type_code(h.dtype), _at(codes),
            _at(scales), _at(slots), n, _at(h))
    return h


@_streamed
def decode_step_cached(codes, scales, slots, x_t, x_prev, B_t, B_prev, C_t, dt, A, lam, theta, *,
                       y=None):
    """One decode step on states in an 8-bit cache, in place
    (m3_decode_step_cached).

    codes [slots,H,N,P] int8 or float8_e4m3fn with scales [slots,H,N]
    float32; slots [S] int32 (idle where negative or past the pool; None:
    sequence i in slot i); the rest as for decode_step.  Returns y [S,H,R,P],
    whose rows of idle entries are left as they were (zeros when y is not
    given)."""
    import torch
    lib = _lib or load_library()
    dev = codes.get_device()
    code = _cache_same(codes, scales, slots, dev)
    n, nh, nn, npd = codes.shape
    ns, nr = x_t.shape[0], x_t.shape[2]
    xs, bs = (ns, nh, nr, npd), (ns, nh, nr, nn)
    tcode = _type_code(x_t.dtype)
    if slots is not None and slots.shape[0] != ns:
        raise ValueError("slots: expected shape %s, got %s" % ((ns,), tuple(slots.shape)))
    if lam is not None and (x_prev is None or B_prev is None):
        raise ValueError("x_prev and B_prev are required with lam")
    for name, t, shape in (("x_t", x_t, xs), ("x_prev", x_prev, xs), ("B_t", B_t, bs),
                           ("B_prev", B_prev, bs), ("C_t", C_t, bs)):
        if t is not None:
            _same(t, name, x_t.dtype, shape, dev)
    _same(dt, "dt", torch.float32, (ns, nh), dev)
    if lam is not None:
        _same(lam, "lam", torch.float32, (ns, nh), dev)
    if theta is not None:
        _same(theta, "theta", torch.float32, (ns, nh, nn // 2), dev)
    _same(A, "A", torch.float32, (nh,), dev)
    if y is not None:
        _same(y, "y", x_t.dtype, xs, dev)
    _gpu(dev)
    if y is None:
        y = (torch.empty if slots is None else torch.zeros)(xs, dtype=x_t.dtype, device=dev)
    d = M3Dims(ns, 1, nh, npd, nn, nr)
    _launch(dev, lib.m3_decode_step_cached, ctypes.byref(d), tcode, code, _at(codes),
            _at(scales), _at(slots), n, _at(x_t), _at(x_prev), _at(B_t), _at(B_prev),
            _at(C_t), _at(dt), _at(A), _at(lam), _at(theta), _at(y))
    return y


_tensors = None


def _look():
    """The module that looks at a call's tensors and makes the new ones (see
    csrc/tensors.cpp); _dense and _spaced say what it found wrong."""
    global _tensors
    if _tensors is None:
        load_library()
        try:
            from . import _tensors as found
        except ImportError as e:
            raise RuntimeError("_tensors.so not found beside libm3ssm.so; build it with "
                               "`python -m state_space_sequence_exp_amd.build`") from e
        _tensors = found
    return _tensors


def _dense(names, dtype, shape, dev: int, *ts):
    """Addresses of dense arrays of this type and shape on device `dev` (None: 0)."""
    got = _tensors.dense(dtype, shape, dev, *ts)
    if got is None:
        for name, t in zip(names, ts):
            if t is not None:
                _same(t, name, dtype, shape, dev)
        raise ValueError("%s: expected dense arrays" % (names,))
    return got


def _spaced(names, dtype, shape, dev: int, *ts):
    """Address and row distance of each of these arrays of rows (None: 0, 0)."""
    got = _tensors.rows(dtype, shape, dev, *ts)
    if got is None:
        for name, t in zip(names, ts):
            if t is not None:
                _rows(t, name, dtype, shape, dev)
        raise ValueError("%s: expected arrays of rows" % (names,))
    return got


@_streamed
def causal_conv(x, weight, bias=None, *, silu: bool = False, state=None, lengths=None, y=None,
                state_out=None, want_state: bool = True) -> Tuple:
    """Short causal convolution over the tokens, one filter of W = 2, 3 or 4 taps
    a channel (m3_causal_conv): y_t = act(bias + sum_k weight[:, k] x_{t-(W-1)+k}),
    act the silu with silu=True, the identity without.

    x [B,T,D] float32 or bfloat16, tokens at one distance (a slice of a wider
    projection is read in place); weight [D,W], bias [D] float32.  state
    [B,W-1,D] in x's type: the inputs before the first token, the oldest first
    (None: zeros).  lengths [B] int32: the tokens of each sequence; those behind
    are padding, not looked at, their y is 0.  y and state_out may be given;
    they must not overlap an input or each other.
    Returns (y, state [B,W-1,D]: the last W-1 inputs, for the next piece or
    causal_conv_step; None without want_state).
    """
    import torch
    _tensors or _look()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if len(shape) != 3:
        raise ValueError("x: expected [B, T, D], got %s" % (tuple(shape),))
    nb, nt, nd = shape
    code = _type_code(dt)
    if weight.dim() != 2:
        raise ValueError("weight: expected [D, W], got %s" % (tuple(weight.shape),))
    nw = weight.shape[1]
    px, ldx, py, ldy = _spaced(("x", "y"), dt, shape, dev, x, y)
    pw, = _dense(("weight",), torch.float32, (nd, nw), dev, weight)
    pb, = _dense(("bias",), torch.float32, (nd,), dev, bias)
    ps, pk = _dense(("state", "state_out"), dt, (nb, nw - 1, nd), dev, state, state_out)
    pl, = _dense(("lengths",), torch.int32, (nb,), dev, lengths)
    _gpu(dev)
    if y is None:
        y = _tensors.empty(dt, shape, x)
        py = y.data_ptr()
    if state_out is None and want_state:
        state_out = _tensors.empty(dt, (nb, nw - 1, nd), x)
        pk = state_out.data_ptr()
    d = M3ConvDims(nb, nt, nd, nw, ldx, ldy)
    _launch(dev, _lib.m3_causal_conv, ctypes.byref(d), code, px, pw, pb, 1 if silu else 0, ps, pl, py, pk)
    return y, state_out


@_streamed
def causal_conv_step(state, x, weight, bias=None, *, silu: bool = False, slots=None, y=None):
    """One token of the short causal convolution, its states updated in place
    (m3_causal_conv_step).

    state [slots,W-1,D] in x's type; x [B,D] float32 or bfloat16; slots [B] int32
    names each row's state (negative, past the pool, or named by a row before:
    idle; None: row b in slot b).  Returns y [B,D], whose idle rows are left as
    they were (zeros when y is not given)."""
    import torch
    _tensors or _look()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if len(shape) != 2:
        raise ValueError("x: expected [B, D], got %s" % (tuple(shape),))
    nb, nd = shape
    code = _type_code(dt)
    if weight.dim() != 2 or state.dim() != 3:
        raise ValueError("expected weight [D, W] and state [slots, W-1, D], got %s and %s"
                         % (tuple(weight.shape), tuple(state.shape)))
    nw, ns = weight.shape[1], state.shape[0]
    px, ldx, py, ldy = _spaced(("x", "y"), dt, shape, dev, x, y)
    pw, = _dense(("weight",), torch.float32, (nd, nw), dev, weight)
    pb, = _dense(("bias",), torch.float32, (nd,), dev, bias)
    ps, = _dense(("state",), dt, (ns, nw - 1, nd), dev, state)
    pi = _pool_slots(slots, nb, ns, dev)
    _gpu(dev)
    if y is None:
        y = _step_output(x, slots)
        py = y.data_ptr()
    d = M3ConvDims(nb, 1, nd, nw, ldx, ldy)
    _launch(dev, _lib.m3_causal_conv_step, ctypes.byref(d), code, ps, pi, ns, px, pw, pb,
            1 if silu else 0, py)
    return y


def _pool_slots(slots, nb, n_slots, dev):
    import torch
    if slots is None:
        if nb > n_slots:
            raise ValueError("%d rows without slots for a pool of %d" % (nb, n_slots))
        return 0
    return _dense(("slots",), torch.int32, (nb,), dev, slots)[0]


def _step_output(x, slots):
    """A single-token call's new y: zeros where rows may be idle."""
    import torch
    if slots is None:
        return _tensors.empty(x.dtype, x.shape, x)
    return torch.zeros(x.shape, dtype=x.dtype, device=x.device)


def selective_scan_workspace_size(batch, seqlen, channels, N, dtype) -> int:
    """Bytes of workspace selective_scan needs (0: none)."""
    d = M3SelectDims(int(batch), int(seqlen), int(channels), int(N))
    return int(load_library().m3_selective_scan_workspace_size(ctypes.byref(d), _type_code(dtype)))


@_streamed
def selective_scan(x, dt, A, B, C, skip=None, z=None, *, dt_bias=None, softplus: bool = True,
                   h0=None, lengths=None, y=None, h_last=None, workspace=None) -> Tuple:
    """Selective state space scan over a sequence (m3_selective_scan): per channel
    N states, s = softplus(dt + dt_bias) (dt + dt_bias with softplus=False),
    h[n] = exp(s A[n]) h[n] + s x B[n], y = (sum_n C[n] h[n] + skip x) silu(z).

    x, dt, z [B,T,D] and B, C [B,T,N], N <= 64, float32 or bfloat16 (one type),
    tokens at one distance in each (slices of wider projections are read in
    place); A [D,N], skip, dt_bias [D] float32; h0 [B,D,N] float32 or None
    (zeros).  lengths [B] int32: the tokens of each sequence; those behind are
    padding, not looked at, their y is 0.  y and h_last may be given; they must
    not overlap an input or each other.  A workspace
    (selective_scan_workspace_size bytes, of any content) may be kept for later
    calls; calls that overlap need distinct ones.
    Returns (y [B,T,D], h_last [B,D,N] float32: each sequence's state after its
    own last token)."""
    import torch
    _tensors or _look()
    shape, dev, dtype = x.shape, x.get_device(), x.dtype
    if len(shape) != 3 or A.dim() != 2:
        raise ValueError("expected x [B, T, D] and A [D, N], got %s and %s"
                         % (tuple(shape), tuple(A.shape)))
    nb, nt, nd = shape
    nn = A.shape[1]
    code = _type_code(dtype)
    px, ldx, pt, ldt, pz, ldz, py, ldy = _spaced(("x", "dt", "z", "y"), dtype, shape, dev, x, dt, z, y)
    pB, ldb, pC, ldc = _spaced(("B", "C"), dtype, (nb, nt, nn), dev, B, C)
    pA, = _dense(("A",), torch.float32, (nd, nn), dev, A)
    pk, pd = _dense(("skip", "dt_bias"), torch.float32, (nd,), dev, skip, dt_bias)
    p0, ph = _dense(("h0", "h_last"), torch.float32, (nb, nd, nn), dev, h0, h_last)
    pl, = _dense(("lengths",), torch.int32, (nb,), dev, lengths)
    _gpu(dev)
    if y is None:
        y = _tensors.empty(dtype, shape, x)
        py = y.data_ptr()
    if h_last is None:
        h_last = _tensors.empty(torch.float32, (nb, nd, nn), x)
        ph = h_last.data_ptr()
    d = M3SelectDims(nb, nt, nd, nn, ldx, ldt, ldz, ldy, ldb, ldc)
    need = _lib.m3_selective_scan_workspace_size(ctypes.byref(d), code)
    pw = ws_bytes = 0
    if need:
        if workspace is None:
            workspace = _tensors.empty(torch.uint8, (need,), x)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the first tensor's device")
        pw, ws_bytes = workspace.data_ptr(), workspace.nbytes
    _launch(dev, _lib.m3_selective_scan, ctypes.byref(d), code, px, pt, pA, pB, pC, pk, pz, pd,
            1 if softplus else 0, p0, pl, py, ph, pw, ws_bytes)
    return y, h_last


@_streamed
def selective_scan_step(h, x, dt, A, B, C, skip=None, z=None, *, dt_bias=None, softplus: bool = True,
                        slots=None, y=None):
    """One token of the selective scan, its states updated in place
    (m3_selective_scan_step).

    h [slots,D,N] float32; x, dt, z [B,D] and B, C [B,N] float32 or bfloat16;
    slots [B] int32 as for causal_conv_step; the rest as for selective_scan.
    Returns y [B,D], whose idle rows are left as they were (zeros when y is not
    given)."""
    import torch
    _tensors or _look()
    shape, dev, dtype = x.shape, x.get_device(), x.dtype
    if len(shape) != 2 or A.dim() != 2 or h.dim() != 3:
        raise ValueError("expected h [slots, D, N], x [B, D] and A [D, N], got %s, %s and %s"
                         % (tuple(h.shape), tuple(shape), tuple(A.shape)))
    nb, nd = shape
    nn, ns = A.shape[1], h.shape[0]
    code = _type_code(dtype)
    px, ldx, pt, ldt, pz, ldz, py, ldy = _spaced(("x", "dt", "z", "y"), dtype, shape, dev, x, dt, z, y)
    pB, ldb, pC, ldc = _spaced(("B", "C"), dtype, (nb, nn), dev, B, C)
    pA, = _dense(("A",), torch.float32, (nd, nn), dev, A)
    ph, = _dense(("h",), torch.float32, (ns, nd, nn), dev, h)
    pk, pd = _dense(("skip", "dt_bias"), torch.float32, (nd,), dev, skip, dt_bias)
    pi = _pool_slots(slots, nb, ns, dev)
    _gpu(dev)
    if y is None:
        y = _step_output(x, slots)
        py = y.data_ptr()
    d = M3SelectDims(nb, 1, nd, nn, ldx, ldt, ldz, ldy, ldb, ldc)
    _launch(dev, _lib.m3_selective_scan_step, ctypes.byref(d), code, ph, pi, ns, px, pt, pA, pB, pC,
            pk, pz, pd, 1 if softplus else 0, py)
    return y


def _ffn_shapes(x, w_gate):
    """Rows, K, F and the shape of h."""
    shape = x.shape
    if len(shape) < 1 or w_gate.dim() != 2:
        raise ValueError("expected x [..., K] and w_gate [F, K], got %s and %s"
                         % (tuple(shape), tuple(w_gate.shape)))
    nf, lead = w_gate.shape[0], shape[:-1]
    return math.prod(lead), shape[-1], nf, (*lead, nf)


@_streamed
def gated_ffn(x, w_gate, w_up, *, want_pre: bool = False, h=None, gate=None, up=None) -> Tuple:
    """Gated feed-forward projections (m3_gated_ffn): h = silu(x w_gate^T) * (x
    w_up^T), both products, the activation and the gate in one kernel.

    x [...,K], w_gate, w_up [F,K] float32 or bfloat16 (one type), rows at one
    distance.  want_pre keeps the two products, in float32, for the backward pass.
    h, gate and up may be given (gate and up together); they must not overlap an
    input or each other.
    Returns (h [...,F], gate, up [...,F] float32 or None)."""
    import torch
    _tensors or _look()
    dev, dt = x.get_device(), x.dtype
    rows, nk, nf, out = _ffn_shapes(x, w_gate)
    code = _type_code(dt)
    px, ldx = _spaced(("x",), dt, x.shape, dev, x)
    pg, ldg, pu, ldu = _spaced(("w_gate", "w_up"), dt, (nf, nk), dev, w_gate, w_up)
    ph, ldh = _spaced(("h",), dt, out, dev, h)
    if (gate is None) != (up is None):
        raise ValueError("gate and up go together")
    qg, lqg, qu, lqu = _spaced(("gate", "up"), torch.float32, out, dev, gate, up)
    _gpu(dev)
    if h is None:
        h = _tensors.empty(dt, out, x)
        ph = h.data_ptr()
    if gate is None and want_pre:
        gate, up = _tensors.empty(torch.float32, out, x), _tensors.empty(torch.float32, out, x)
        qg, qu = gate.data_ptr(), up.data_ptr()
    d = M3FfnDims(rows, nk, nf, ldx, ldg, ldu, ldh, lqg, lqu)
    _launch(dev, _lib.m3_gated_ffn, ctypes.byref(d), code, px, pg, pu, ph, qg, qu)
    return h, gate, up


def gated_ffn_backward_workspace_size(rows, channels, hidden, dtype) -> int:
    """Bytes of workspace gated_ffn_backward needs (0 for no rows)."""
    d = M3FfnDims(int(rows), int(channels), int(hidden))
    return int(load_library().m3_gated_ffn_backward_workspace_size(ctypes.byref(d), _type_code(dtype)))


@_streamed
def gated_ffn_backward(dh, x, w_gate, w_up, gate, up, *, dx=None, dw_gate=None, dw_up=None,
                       want_x: bool = True, want_weights: bool = True, workspace=None):
    """Gradients of sum(h * dh) for gated_ffn's inputs (m3_gated_ffn_backward);
    gate and up as gated_ffn kept them.  dx, dw_gate and dw_up may be given (the
    last two together).  A workspace (gated_ffn_backward_workspace_size bytes, of
    any content) may be kept for later calls; calls that overlap need distinct
    ones.  Returns a dict: x (absent without want_x), w_gate and w_up (absent
    without want_weights) in the inputs' type."""
    import torch
    _tensors or _look()
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    rows, nk, nf, out = _ffn_shapes(x, w_gate)
    code = _type_code(dt)
    if (dw_gate is None) != (dw_up is None):
        raise ValueError("dw_gate and dw_up go together")
    if (dx is not None and not want_x) or (dw_gate is not None and not want_weights):
        raise ValueError("a gradient that is given is wanted")
    px, ldx, pdx, lddx = _spaced(("x", "dx"), dt, shape, dev, x, dx)
    pg, ldg, pu, ldu, pdg, lddg, pdu, lddu = _spaced(("w_gate", "w_up", "dw_gate", "dw_up"), dt, (nf, nk), dev,
                                                     w_gate, w_up, dw_gate, dw_up)
    qg, lqg, qu, lqu = _spaced(("gate", "up"), torch.float32, out, dev, gate, up)
    pdh, lddh = _spaced(("dh",), dt, out, dev, dh)
    _gpu(dev)
    if dx is None and want_x:
        dx = _tensors.empty(dt, shape, x)
        pdx = dx.data_ptr()
    if dw_gate is None and want_weights:
        dw_gate, dw_up = _tensors.empty(dt, (nf, nk), x), _tensors.empty(dt, (nf, nk), x)
        pdg, pdu = dw_gate.data_ptr(), dw_up.data_ptr()
    d = M3FfnDims(rows, nk, nf, ldx, ldg, ldu, 0, lqg, lqu, lddh, lddx, lddg, lddu)
    need = _lib.m3_gated_ffn_backward_workspace_size(ctypes.byref(d), code)
    if workspace is None and need:
        workspace = _tensors.empty(torch.uint8, (need,), x)
    elif workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the first tensor's device")
    pw, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _launch(dev, _lib.m3_gated_ffn_backward, ctypes.byref(d), code, pdh, px, pg, pu, qg, qu, pdx, pdg, pdu,
            pw, ws_bytes)
    res = {}
    if dx is not None:
        res["x"] = dx
    if dw_gate is not None:
        res["w_gate"], res["w_up"] = dw_gate, dw_up
    return res
