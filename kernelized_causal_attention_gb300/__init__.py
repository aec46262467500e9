"""GB300 (sm_103a) elu(x)+1 linear attention: Python binding of the C ABI.

This module only marshals arguments: it loads ``_lib/liblinattn.so`` (built by
``_build.py``), passes tensor data pointers and the current CUDA stream to the
C entry points declared in ``include/linattn.h``, and turns error codes into
exceptions.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback of any kind, and using any entry point without
the built library raises.

Raw entry points (same names and argument order as the C ABI, tensors in
place of pointers): ``la_causal_fwd``, ``la_causal_bwd``, ``la_causal_prefill``,
``la_noncausal_fwd``, ``la_noncausal_bwd``, ``la_decode_step``, the decayed
``la_causal_fwd_decay``, ``la_causal_bwd_decay``, ``la_decode_step_decay``, the projected
``la_decode_step_proj``, the degree-2 polynomial ``la_causal_fwd_poly``,
``la_causal_bwd_poly``, the short convolution's ``la_short_conv_fwd``, ``la_short_conv_bwd``,
``la_short_conv_step``, the selective scan's ``la_scan_fwd``, ``la_scan_bwd``, ``la_scan_step``, the cross
attention's ``la_cross_fwd``, ``la_cross_bwd``, ``la_cross_step``, ``la_workspace_bytes``, ``la_device_status``.
Convenience wrappers that allocate outputs with torch: ``causal_fwd``,
``causal_bwd``, ``causal_prefill``, ``noncausal_fwd``, ``noncausal_bwd``, ``decode_step``, ``decode_step_proj``,
``causal_fwd_poly``, ``causal_bwd_poly``, ``short_conv_fwd``, ``short_conv_bwd``, ``short_conv_step``,
``scan_fwd``, ``scan_bwd``, ``scan_step``, ``cross_fwd``, ``cross_bwd``, ``cross_step`` and the
autograd functions ``causal_linear_attention`` / ``noncausal_linear_attention`` /
``short_conv`` / ``selective_scan`` / ``cross_linear_attention``.

The method is Katharopoulos et al., "Transformers are RNNs" (part 2/3):
eq. 7 (phi), §3.3 eq. 9-12, §3.3.1 eq. 13-15, §3.4 eq. 16-20.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "liblinattn.so")

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA, LA_ERR_TIMEOUT, LA_ERR_WORKSPACE = range(6)
LA_F32, LA_BF16 = 0, 1
(LA_OP_CAUSAL_FWD, LA_OP_CAUSAL_BWD, LA_OP_NONCAUSAL_FWD, LA_OP_NONCAUSAL_BWD, LA_OP_DECODE,
 LA_OP_CAUSAL_PREFILL, LA_OP_CAUSAL_FWD_DECAY, LA_OP_CAUSAL_BWD_DECAY, LA_OP_DECODE_PROJ,
 LA_OP_CAUSAL_FWD_POLY, LA_OP_CAUSAL_BWD_POLY) = range(11)

# exported symbols and their ctypes signatures ("p" pointer, "i" int, "z" size_t,
# "u" unsigned long long)
_SIGS = {
    "la_status_string": ("i", ctypes.c_char_p),
    "la_version": ("", ctypes.c_int),
    "la_workspace_bytes": ("i i i i i i i", ctypes.c_size_t),
    "la_kernel_launches": ("i i i i i i i", ctypes.c_int),
    "la_causal_fwd": ("p p p p p p z i i i i i i p", ctypes.c_int),
    "la_causal_bwd": ("p p p p p p p p p p z i i i i i i p", ctypes.c_int),
    "la_causal_prefill": ("p p p p p p p p z i i i i i i p", ctypes.c_int),
    "la_noncausal_fwd": ("p p p p p p p p p z i i i i i i p", ctypes.c_int),
    "la_noncausal_bwd": ("p p p p p p p p p p p p p z i i i i i i p", ctypes.c_int),
    "la_decode_step": ("p p p p p p i i i i i p", ctypes.c_int),
    "la_causal_fwd_decay": ("p p p p p f p z i i i i i i p", ctypes.c_int),
    "la_causal_bwd_decay": ("p p p p p p p p p f p z i i i i i i p", ctypes.c_int),
    "la_decode_step_decay": ("p p p p p p f i i i i i p", ctypes.c_int),
    "la_decode_step_proj": ("p p p p p i i i i i i p", ctypes.c_int),
    "la_causal_fwd_poly": ("p p p p p p z i i i i i i p", ctypes.c_int),
    "la_causal_bwd_poly": ("p p p p p p p p p p z i i i i i i p", ctypes.c_int),
    "la_causal_fwd_noalloc": ("p p p p p i i i i i i p", ctypes.c_int),
    "la_short_conv_workspace_bytes": ("i i i i i", ctypes.c_size_t),
    "la_short_conv_fwd": ("p p p p p p i i i i i i i p", ctypes.c_int),
    "la_short_conv_bwd": ("p p p p p p p p p z i i i i i i i p", ctypes.c_int),
    "la_short_conv_step": ("p p p p p i i i i i i p", ctypes.c_int),
    "la_scan_workspace_bytes": ("i i i i i i i i", ctypes.c_size_t),
    "la_scan_fwd": ("p p p p p p p p p p p z i i i i i i i i i i i p", ctypes.c_int),
    "la_scan_bwd": ("p p p p p p p p p p p p p p p p p z i i i i i i i i i i i p", ctypes.c_int),
    "la_scan_step": ("p p p p p p p p p i i i i i i i i i i p", ctypes.c_int),
    "la_cross_workspace_bytes": ("i i i i i i i i i", ctypes.c_size_t),
    "la_cross_fwd": ("p p p p p p p p p z i i i i i i i i p", ctypes.c_int),
    "la_cross_bwd": ("p p p p p p p p p p p p p z i i i i i i i i p", ctypes.c_int),
    "la_cross_step": ("p p p p i i i i i i p", ctypes.c_int),
    "la_device_status": ("p i p", ctypes.c_int),
    "la_selftest_wait": ("p u", ctypes.c_int),
}
EXPORTED = tuple(_SIGS)

_lock = threading.Lock()
_lib = None


class LinAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (code {code})")


def library_path() -> str:
    return LIB_PATH


def lib():
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library not built: {LIB_PATH} is missing. Build it with "
                    "`python -m kernelized_causal_attention_gb300._build` (needs nvcc).")
            h = ctypes.CDLL(LIB_PATH)
            kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int, "z": ctypes.c_size_t,
                     "u": ctypes.c_ulonglong, "f": ctypes.c_float}
            for name, (sig, res) in _SIGS.items():
                fn = getattr(h, name)
                fn.argtypes = [kinds[c] for c in sig.split()]
                fn.restype = res
            _lib = h
    return _lib


def status_string(code: int) -> str:
    return lib().la_status_string(int(code)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use float32 or bfloat16")


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)  # a raw address
    if not t.is_cuda:
        # the library takes device pointers; a host address would reach a kernel
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _pv(t):
    """A device address without the contiguity check (row-strided inputs)."""
    if isinstance(t, torch.Tensor):
        if not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device")
        return t.data_ptr()
    return t


def _current_stream():
    """The current device's current stream as an address."""
    return torch.cuda.current_stream().cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same address without building a Stream object (3 us)
    def _current_stream():  # noqa: F811
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(rc: int, where: str):
    if rc != LA_OK:
        raise LinAttnError(rc, where)


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


# ------------------------------------------------------------------ raw C ABI

def la_workspace_bytes(op, B, H, N, D, M, dtype) -> int:
    return int(lib().la_workspace_bytes(op, B, H, N, D, M, dtype))


def la_kernel_launches(op, B, H, N, D, M, dtype) -> int:
    return int(lib().la_kernel_launches(op, B, H, N, D, M, dtype))


def la_causal_fwd(q, k, v, out, den, workspace, B, H, N, D, M, dtype, stream=None):
    _check(lib().la_causal_fwd(_p(q), _p(k), _p(v), _p(out), _p(den), _p(workspace),
                               _nbytes(workspace), B, H, N, D, M, dtype, _stream(stream)),
           "la_causal_fwd")


def la_causal_bwd(q, k, v, out, den, dout, dq, dk, dv, workspace, B, H, N, D, M, dtype,
                  stream=None):
    _check(lib().la_causal_bwd(_p(q), _p(k), _p(v), _p(out), _p(den), _p(dout), _p(dq), _p(dk),
                               _p(dv), _p(workspace), _nbytes(workspace), B, H, N, D, M, dtype,
                               _stream(stream)), "la_causal_bwd")


def la_causal_prefill(q, k, v, out, den, S, Z, workspace, B, H, N, D, M, dtype, stream=None):
    _check(lib().la_causal_prefill(_p(q), _p(k), _p(v), _p(out), _p(den), _p(S), _p(Z),
                                   _p(workspace), _nbytes(workspace), B, H, N, D, M, dtype,
                                   _stream(stream)), "la_causal_prefill")


def la_noncausal_fwd(q, k, v, lengths, out, den, S, Z, workspace, B, H, N, D, M, dtype,
                     stream=None):
    _check(lib().la_noncausal_fwd(_p(q), _p(k), _p(v), _p(lengths), _p(out), _p(den), _p(S),
                                  _p(Z), _p(workspace), _nbytes(workspace), B, H, N, D, M, dtype,
                                  _stream(stream)), "la_noncausal_fwd")


def la_noncausal_bwd(q, k, v, lengths, out, den, S, Z, dout, dq, dk, dv, workspace, B, H, N, D,
                     M, dtype, stream=None):
    _check(lib().la_noncausal_bwd(_p(q), _p(k), _p(v), _p(lengths), _p(out), _p(den), _p(S),
                                  _p(Z), _p(dout), _p(dq), _p(dk), _p(dv), _p(workspace),
                                  _nbytes(workspace), B, H, N, D, M, dtype, _stream(stream)),
           "la_noncausal_bwd")


def la_decode_step(q, k, v, S, Z, y, B, H, D, M, dtype, stream=None):
    _check(lib().la_decode_step(_p(q), _p(k), _p(v), _p(S), _p(Z), _p(y), B, H, D, M, dtype,
                                _stream(stream)), "la_decode_step")


def la_causal_fwd_decay(q, k, v, out, den, gamma, workspace, B, H, N, D, M, dtype, stream=None):
    _check(lib().la_causal_fwd_decay(_p(q), _p(k), _p(v), _p(out), _p(den), float(gamma),
                                     _p(workspace), _nbytes(workspace), B, H, N, D, M, dtype,
                                     _stream(stream)), "la_causal_fwd_decay")


def la_causal_bwd_decay(q, k, v, out, den, dout, dq, dk, dv, gamma, workspace, B, H, N, D, M,
                        dtype, stream=None):
    _check(lib().la_causal_bwd_decay(_p(q), _p(k), _p(v), _p(out), _p(den), _p(dout), _p(dq),
                                     _p(dk), _p(dv), float(gamma), _p(workspace),
                                     _nbytes(workspace), B, H, N, D, M, dtype, _stream(stream)),
           "la_causal_bwd_decay")


def la_decode_step_decay(q, k, v, S, Z, y, gamma, B, H, D, M, dtype, stream=None):
    _check(lib().la_decode_step_decay(_p(q), _p(k), _p(v), _p(S), _p(Z), _p(y), float(gamma), B,
                                      H, D, M, dtype, _stream(stream)), "la_decode_step_decay")


def la_causal_fwd_poly(q, k, v, out, den, workspace, B, H, N, D, M, dtype, stream=None):
    _check(lib().la_causal_fwd_poly(_p(q), _p(k), _p(v), _p(out), _p(den), _p(workspace),
                                    _nbytes(workspace), B, H, N, D, M, dtype, _stream(stream)),
           "la_causal_fwd_poly")


def la_causal_bwd_poly(q, k, v, out, den, dout, dq, dk, dv, workspace, B, H, N, D, M, dtype,
                       stream=None):
    _check(lib().la_causal_bwd_poly(_p(q), _p(k), _p(v), _p(out), _p(den), _p(dout), _p(dq), _p(dk),
                                    _p(dv), _p(workspace), _nbytes(workspace), B, H, N, D, M, dtype,
                                    _stream(stream)), "la_causal_bwd_poly")


def la_decode_step_proj(x, W, S, Z, y, B, H, d_model, D, M, dtype, stream=None):
    _check(lib().la_decode_step_proj(_p(x), _p(W), _p(S), _p(Z), _p(y), B, H, d_model, D, M, dtype,
                                     _stream(stream)), "la_decode_step_proj")


def la_causal_fwd_noalloc(q, k, v, out, den, B, H, N, D, M, dtype, stream=None):
    """la_causal_fwd with the library's built-in scratch instead of a workspace
    (for callers that may not allocate device memory)."""
    _check(lib().la_causal_fwd_noalloc(_p(q), _p(k), _p(v), _p(out), _p(den), B, H, N, D, M,
                                       dtype, _stream(stream)), "la_causal_fwd_noalloc")


def la_short_conv_workspace_bytes(B, N, C, K, dtype) -> int:
    return int(lib().la_short_conv_workspace_bytes(B, N, C, K, dtype))


def la_short_conv_fwd(x, w, bias, lengths, state, y, B, N, C, K, ldx, silu, dtype, stream=None):
    _check(lib().la_short_conv_fwd(_pv(x), _p(w), _p(bias), _p(lengths), _p(state), _p(y), B, N, C,
                                   K, ldx, int(silu), dtype, _stream(stream)), "la_short_conv_fwd")


def la_short_conv_bwd(x, w, bias, lengths, dy, dx, dw, db, workspace, B, N, C, K, ldx, silu, dtype,
                      stream=None):
    _check(lib().la_short_conv_bwd(_pv(x), _p(w), _p(bias), _p(lengths), _p(dy), _p(dx), _p(dw),
                                   _p(db), _p(workspace), _nbytes(workspace), B, N, C, K, ldx,
                                   int(silu), dtype, _stream(stream)), "la_short_conv_bwd")


def la_short_conv_step(x, w, bias, state, y, B, C, K, ldx, silu, dtype, stream=None):
    _check(lib().la_short_conv_step(_pv(x), _p(w), _p(bias), _p(state), _p(y), B, C, K, ldx,
                                    int(silu), dtype, _stream(stream)), "la_short_conv_step")


def la_scan_workspace_bytes(bwd, B, H, G, N, D, M, dtype) -> int:
    return int(lib().la_scan_workspace_bytes(int(bwd), B, H, G, N, D, M, dtype))


def la_scan_fwd(x, dt, A, Bm, Cm, skip, dt_bias, lengths, S, y, workspace, B, H, G, N, D, M, ldx,
                lddt, ldb, ldc, dtype, stream=None):
    _check(lib().la_scan_fwd(_pv(x), _pv(dt), _p(A), _pv(Bm), _pv(Cm), _p(skip), _p(dt_bias),
                             _p(lengths), _p(S), _p(y), _p(workspace), _nbytes(workspace), B, H, G,
                             N, D, M, ldx, lddt, ldb, ldc, dtype, _stream(stream)), "la_scan_fwd")


def la_scan_bwd(x, dt, A, Bm, Cm, skip, dt_bias, lengths, dy, dx, ddt, dA, dB, dC, dskip, ddt_bias,
                workspace, B, H, G, N, D, M, ldx, lddt, ldb, ldc, dtype, stream=None):
    _check(lib().la_scan_bwd(_pv(x), _pv(dt), _p(A), _pv(Bm), _pv(Cm), _p(skip), _p(dt_bias),
                             _p(lengths), _p(dy), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC),
                             _p(dskip), _p(ddt_bias), _p(workspace), _nbytes(workspace), B, H, G, N,
                             D, M, ldx, lddt, ldb, ldc, dtype, _stream(stream)), "la_scan_bwd")


def la_scan_step(x, dt, A, Bm, Cm, skip, dt_bias, S, y, B, H, G, D, M, ldx, lddt, ldb, ldc, dtype,
                 stream=None):
    _check(lib().la_scan_step(_pv(x), _pv(dt), _p(A), _pv(Bm), _pv(Cm), _p(skip), _p(dt_bias), _p(S),
                              _p(y), B, H, G, D, M, ldx, lddt, ldb, ldc, dtype, _stream(stream)),
           "la_scan_step")


def la_cross_workspace_bytes(bwd, B, H, Hk, Nq, Nk, D, M, dtype) -> int:
    return int(lib().la_cross_workspace_bytes(int(bwd), B, H, Hk, Nq, Nk, D, M, dtype))


def la_cross_fwd(q, k, v, lengths, out, den, S, Z, workspace, B, H, Hk, Nq, Nk, D, M, dtype,
                 stream=None):
    _check(lib().la_cross_fwd(_p(q), _p(k), _p(v), _p(lengths), _p(out), _p(den), _p(S), _p(Z),
                              _p(workspace), _nbytes(workspace), B, H, Hk, Nq, Nk, D, M, dtype,
                              _stream(stream)), "la_cross_fwd")


def la_cross_bwd(q, k, v, lengths, out, den, S, Z, dout, dq, dk, dv, workspace, B, H, Hk, Nq, Nk, D,
                 M, dtype, stream=None):
    _check(lib().la_cross_bwd(_p(q), _p(k), _p(v), _p(lengths), _p(out), _p(den), _p(S), _p(Z),
                              _p(dout), _p(dq), _p(dk), _p(dv), _p(workspace), _nbytes(workspace), B,
                              H, Hk, Nq, Nk, D, M, dtype, _stream(stream)), "la_cross_bwd")


def la_cross_step(q, S, Z, y, B, H, Hk, D, M, dtype, stream=None):
    _check(lib().la_cross_step(_p(q), _p(S), _p(Z), _p(y), B, H, Hk, D, M, dtype, _stream(stream)),
           "la_cross_step")


def la_device_status(clear=True, stream=None):
    """(status, code): LA_OK and 0, or LA_ERR_TIMEOUT and the code of the first
    bounded wait inside a kernel that ran out (after the stream's queued work);
    clear resets the status word."""
    code = ctypes.c_int(0)
    rc = lib().la_device_status(_stream(stream), int(bool(clear)), ctypes.byref(code))
    if rc not in (LA_OK, LA_ERR_TIMEOUT):
        raise LinAttnError(rc, "la_device_status")
    return rc, code.value


def la_selftest_wait(limit_ns, stream=None):
    """Launches the diagnostic kernel whose bounded wait runs out after limit_ns."""
    _check(lib().la_selftest_wait(_stream(stream), int(limit_ns)), "la_selftest_wait")


def check_device_status(stream=None):
    """Raises LinAttnError(LA_ERR_TIMEOUT) if a kernel's bounded wait ran out
    (and clears the status word); returns None otherwise."""
    rc, code = la_device_status(True, stream)
    if rc != LA_OK:
        raise LinAttnError(rc, f"device status (wait code {code})")


# --------------------------------------------------- allocating convenience API

def workspace(op, B, H, N, D, M, dtype, device):
    n = la_workspace_bytes(op, B, H, N, D, M, dtype)
    return None if n == 0 else torch.empty(n, dtype=torch.uint8, device=device)


def causal_fwd(q, k, v, stream=None):
    """(out, den) of the causal form; q, k [B,H,N,D], v [B,H,N,M] on the GPU."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    out = torch.empty(B, H, N, M, dtype=q.dtype, device=q.device)
    den = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    ws = workspace(LA_OP_CAUSAL_FWD, B, H, N, D, M, dt, q.device)
    la_causal_fwd(q, k, v, out, den, ws, B, H, N, D, M, dt, stream)
    return out, den


def causal_fwd_decay(q, k, v, gamma, stream=None):
    """(out, den) of the causal form with the RetNet decay gamma in [0, 1]."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    out = torch.empty(B, H, N, M, dtype=q.dtype, device=q.device)
    den = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    ws = workspace(LA_OP_CAUSAL_FWD_DECAY, B, H, N, D, M, dt, q.device)
    la_causal_fwd_decay(q, k, v, out, den, gamma, ws, B, H, N, D, M, dt, stream)
    return out, den


def causal_bwd_decay(q, k, v, out, den, dout, gamma, stream=None):
    """(dq, dk, dv) of sum(dout * out) for the decayed causal form."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = workspace(LA_OP_CAUSAL_BWD_DECAY, B, H, N, D, M, dt, q.device)
    la_causal_bwd_decay(q, k, v, out, den, dout, dq, dk, dv, gamma, ws, B, H, N, D, M, dt, stream)
    return dq, dk, dv


def causal_fwd_poly(q, k, v, stream=None):
    """(out, den) of causal attention with the degree-2 polynomial kernel
    sim = (q . k)^2 (bf16, D <= 10)."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    out = torch.empty(B, H, N, M, dtype=q.dtype, device=q.device)
    den = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    ws = workspace(LA_OP_CAUSAL_FWD_POLY, B, H, N, D, M, dt, q.device)
    la_causal_fwd_poly(q, k, v, out, den, ws, B, H, N, D, M, dt, stream)
    return out, den


def causal_bwd_poly(q, k, v, out, den, dout, stream=None):
    """(dq, dk, dv) of sum(dout * out) with the degree-2 polynomial kernel."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = workspace(LA_OP_CAUSAL_BWD_POLY, B, H, N, D, M, dt, q.device)
    la_causal_bwd_poly(q, k, v, out, den, dout, dq, dk, dv, ws, B, H, N, D, M, dt, stream)
    return dq, dk, dv


def decode_step_decay(q, k, v, S, Z, gamma, stream=None):
    """One decayed RNN step; S, Z updated in place.  Returns y [B,H,M]."""
    B, H, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    y = torch.empty(B, H, M, dtype=q.dtype, device=q.device)
    la_decode_step_decay(q, k, v, S, Z, y, gamma, B, H, D, M, dt, stream)
    return y


def causal_prefill(q, k, v, S=None, Z=None, stream=None):
    """(out, den, S, Z): the causal form started from the state (S, Z) (zeros
    if None), which is updated in place to the state after the sequence and
    returned; la_decode_step continues from it."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    out = torch.empty_like(v)
    den = torch.empty(B, H, N, device=q.device, dtype=torch.float32)
    if S is None:
        S = torch.zeros(B, H, D, M, device=q.device, dtype=torch.float32)
    if Z is None:
        Z = torch.zeros(B, H, D, device=q.device, dtype=torch.float32)
    ws = workspace(LA_OP_CAUSAL_PREFILL, B, H, N, D, M, dt, q.device)
    la_causal_prefill(q, k, v, out, den, S, Z, ws, B, H, N, D, M, dt, stream)
    return out, den, S, Z


def causal_bwd(q, k, v, out, den, dout, stream=None):
    """(dq, dk, dv) of sum(dout * out) for the causal form."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = workspace(LA_OP_CAUSAL_BWD, B, H, N, D, M, dt, q.device)
    la_causal_bwd(q, k, v, out, den, dout, dq, dk, dv, ws, B, H, N, D, M, dt, stream)
    return dq, dk, dv


def noncausal_fwd(q, k, v, lengths=None, stream=None):
    """(out, den, S, Z) of the non-causal form; lengths: int32 [B] on the GPU or None."""
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    out = torch.empty(B, H, N, M, dtype=q.dtype, device=q.device)
    den = torch.empty(B, H, N, dtype=torch.float32, device=q.device)
    S = torch.empty(B, H, D, M, dtype=torch.float32, device=q.device)
    Z = torch.empty(B, H, D, dtype=torch.float32, device=q.device)
    ws = workspace(LA_OP_NONCAUSAL_FWD, B, H, N, D, M, dt, q.device)
    la_noncausal_fwd(q, k, v, lengths, out, den, S, Z, ws, B, H, N, D, M, dt, stream)
    return out, den, S, Z


def noncausal_bwd(q, k, v, lengths, out, den, S, Z, dout, stream=None):
    B, H, N, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = workspace(LA_OP_NONCAUSAL_BWD, B, H, N, D, M, dt, q.device)
    la_noncausal_bwd(q, k, v, lengths, out, den, S, Z, dout, dq, dk, dv, ws, B, H, N, D, M, dt,
                     stream)
    return dq, dk, dv


def decode_step(q, k, v, S, Z, stream=None):
    """One RNN step; S [B,H,D,M] and Z [B,H,D] (float32) are updated in place.
    Returns y [B,H,M]."""
    B, H, D = q.shape
    M = v.shape[-1]
    dt = _dtype_code(q)
    y = torch.empty(B, H, M, dtype=q.dtype, device=q.device)
    la_decode_step(q, k, v, S, Z, y, B, H, D, M, dt, stream)
    return y


def decode_step_proj(x, W, S, Z, H, D, M, stream=None):
    """One RNN step whose q, k, v are the projection x W (bf16): x [B, d_model],
    W [d_model, H*(2D+M)] with each head's W_Q | W_K | W_V columns side by side,
    head after head.  S [B,H,D,M] and Z [B,H,D] (float32) are updated in place.
    Returns y [B,H,M] (bf16)."""
    B, dm = x.shape
    y = torch.empty(B, H, M, dtype=x.dtype, device=x.device)
    la_decode_step_proj(x, W, S, Z, y, B, H, dm, D, M, _dtype_code(x), stream)
    return y


# ------------------------- the layer with a data-dependent decay, and its encoder
#
# These wrappers check shapes, types and devices, allocate on the inputs' device and run on that
# device's current stream (``with torch.cuda.stream(s):`` for another one).  A step's kernels take a
# few microseconds, so they are written to cost the host little more than the call itself.

def _take(t, name, shape, dtype, device):
    """The address of a dense tensor of the shape, type and device that the call needs."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise _refusal(t, name, shape, dtype, device)


def _refusal(t, name, shape, dtype, device):
    """What is wrong with a tensor that _take or _take_rows has refused."""
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{name}: a tensor is needed")
    if tuple(t.shape) != tuple(shape):
        return ValueError(f"{name}: shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    if t.dtype != dtype:
        return TypeError(f"{name}: {t.dtype}, the call needs {dtype}")
    if t.device != device:
        return ValueError(f"{name}: on {t.device}, the call is on {device}")
    return ValueError(f"{name}: must be contiguous")


def _take_opt(t, name, shape, dtype, device):
    return None if t is None else _take(t, name, shape, dtype, device)


_INT = (1 << 31) - 1  # the interface's sizes and strides


def _need_ints(*tensors):
    """No size is beyond the interface's integers (only a tensor of as many elements can have one)."""
    for t in tensors:
        if t.numel() > _INT and max(t.shape) > _INT:
            raise ValueError(f"sizes above {_INT}")


def _take_rows(t, name, shape, dtype, device, lead):
    """(address, row stride) of a token-major view whose first `lead` dimensions are batch (and row):
    rows dense, and all rows of all batch entries evenly spaced."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == device):
        raise _refusal(t, name, shape, dtype, device)
    st = t.stride()
    want = shape[-1]
    if len(shape) == lead:
        want = 1
    elif want != 1 and st[-1] != 1:
        raise ValueError(f"{name}: every row must be dense")
    if len(shape) == lead + 2:
        if shape[lead] != 1 and st[lead] != want:
            raise ValueError(f"{name}: every row must be dense")
        want *= shape[lead]
    B = shape[0]
    if lead == 1:
        ld = st[0] if B > 1 else want
    else:
        N = shape[1]
        ld = st[1] if N > 1 else (st[0] if B > 1 else want)
        if B > 1 and st[0] != N * ld:
            raise ValueError(f"{name}: batch entries must be N rows apart")
    if ld > _INT:
        raise ValueError(f"{name}: rows {ld} elements apart, at most {_INT}")
    return t.data_ptr(), ld


def _on_device(f):
    """f with the device of its first argument (given by position or by name) as the current one."""
    first = next(iter(inspect.signature(f).parameters))

    @functools.wraps(f)
    def call(*args, **kw):
        x = args[0] if args else kw.get(first)
        if not isinstance(x, torch.Tensor) or not x.is_cuda or x.get_device() == torch.cuda.current_device():
            return f(*args, **kw)
        with torch.cuda.device(x.device):
            return f(*args, **kw)
    return call


def _need_cuda(t):
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")


def _scratch(n, like):
    """(workspace or None, its address, its size)"""
    if n == 0:
        return None, None, 0
    ws = torch.empty((n,), dtype=torch.uint8, device=like.device)
    return ws, ws.data_ptr(), n


def _conv_args(x, w, bias, lengths, lead):
    if x.dim() != lead + 1 or w.dim() != 2:
        raise ValueError(f"x: {lead + 1} dimensions, w: [C, K]")
    shape, dtype, dev = x.shape, x.dtype, x.device
    C, K = shape[-1], w.shape[1]
    _need_ints(x, w)
    code = _dtype_code(x)
    px, ld = _take_rows(x, "x", shape, dtype, dev, lead)
    pw = _take(w, "w", (C, K), dtype, dev)
    pb = _take_opt(bias, "bias", (C,), dtype, dev)
    pn = _take_opt(lengths, "lengths", shape[:1], torch.int32, dev)
    return shape, C, K, code, dtype, dev, px, ld, pw, pb, pn


@_on_device
def short_conv_fwd(x, w, bias=None, state=None, lengths=None, silu=True):
    """y [B,N,C] of the short causal depthwise convolution: x [B,N,C] (rows may be slices of wider
    ones), w [C,K], K = 2..4, bias [C]; state [B,K-1,C] holds the inputs before row 0 (zeros if None)
    and is updated in place; lengths: int32 [B] of valid rows."""
    (B, N, _), C, K, code, dtype, dev, px, ld, pw, pb, pn = _conv_args(x, w, bias, lengths, 2)
    ps = _take_opt(state, "state", (B, K - 1, C), dtype, dev)
    _need_cuda(x)
    y = torch.empty((B, N, C), dtype=dtype, device=dev)
    _check(lib().la_short_conv_fwd(px, pw, pb, pn, ps, y.data_ptr(), B, N, C, K, ld, int(silu), code, _stream(None)),
           "la_short_conv_fwd")
    return y


@_on_device
def short_conv_bwd(x, w, bias, dy, lengths=None, silu=True):
    """(dx, dw, db) of sum(dy * y) for a history of zeros; db is None without a bias."""
    shape, C, K, code, dtype, dev, px, ld, pw, pb, pn = _conv_args(x, w, bias, lengths, 2)
    B, N, _ = shape
    pg = _take(dy, "dy", shape, dtype, dev)
    _need_cuda(x)
    dx, dw = torch.empty((B, N, C), dtype=dtype, device=dev), torch.empty_like(w)
    db = None if bias is None else torch.empty_like(bias)
    ws, pws, nws = _scratch(lib().la_short_conv_workspace_bytes(B, N, C, K, code), x)
    _check(lib().la_short_conv_bwd(px, pw, pb, pn, pg, dx.data_ptr(), dw.data_ptr(), None if db is None else db.data_ptr(),
                                   pws, nws, B, N, C, K, ld, int(silu), code, _stream(None)), "la_short_conv_bwd")
    return dx, dw, db


@_on_device
def short_conv_step(x, w, bias, state, silu=True):
    """y [B,C] for one row x [B,C] of each stream; state [B,K-1,C] is shifted in place."""
    (B, _), C, K, code, dtype, dev, px, ld, pw, pb, _ = _conv_args(x, w, bias, None, 1)
    ps = _take(state, "state", (B, K - 1, C), dtype, dev)
    _need_cuda(x)
    y = torch.empty((B, C), dtype=dtype, device=dev)
    _check(lib().la_short_conv_step(px, pw, pb, ps, y.data_ptr(), B, C, K, ld, int(silu), code, _stream(None)),
           "la_short_conv_step")
    return y


def _scan_args(x, dt, A, Bm, Cm, skip, dt_bias, lengths, lead):
    """(pointers up to lengths, row strides, sizes (H, G, D, M), type code, type, device)."""
    if x.dim() != lead + 2 or Bm.dim() != lead + 2:
        raise ValueError(f"x, Bm and Cm: {lead + 2} dimensions")
    shape, gshape, dtype, dev = x.shape, Bm.shape, x.dtype, x.device
    rows = shape[:lead]
    H, M, G, D = shape[lead], shape[lead + 1], gshape[lead], gshape[lead + 1]
    _need_ints(x, Bm)
    code = _dtype_code(x)
    px, lx = _take_rows(x, "x", shape, dtype, dev, lead)
    pt, lt = _take_rows(dt, "dt", rows + (H,), dtype, dev, lead)
    pb, lb = _take_rows(Bm, "Bm", rows + (G, D), dtype, dev, lead)
    pc, lc = _take_rows(Cm, "Cm", rows + (G, D), dtype, dev, lead)
    h = (H,)
    ptrs = (px, pt, _take(A, "A", h, dtype, dev), pb, pc, _take_opt(skip, "skip", h, dtype, dev),
            _take_opt(dt_bias, "dt_bias", h, dtype, dev), _take_opt(lengths, "lengths", rows[:1], torch.int32, dev))
    return ptrs, (lx, lt, lb, lc), (H, G, D, M), code, dtype, dev


@_on_device
def scan_fwd(x, dt, A, Bm, Cm, skip=None, dt_bias=None, S=None, lengths=None):
    """y [B,N,H,M] of the selective scan S_n = exp(delta_n A) S_{n-1} + B_n (delta_n x_n)^T,
    y_n = S_n^T C_n + skip x_n, delta = softplus(dt + dt_bias).  x [B,N,H,M], dt [B,N,H], Bm and Cm
    [B,N,G,D] (G divides H; rows may be slices of wider ones), A, skip, dt_bias [H].  S [B,H,D,M]
    (float32) is the state before row 0 (zeros if None), updated in place to the state after each
    sequence's last valid row; scan_step continues from it."""
    ptrs, ld, (H, G, D, M), code, dtype, dev = _scan_args(x, dt, A, Bm, Cm, skip, dt_bias, lengths, 2)
    B, N = x.shape[:2]
    pS = _take_opt(S, "S", (B, H, D, M), torch.float32, dev)
    _need_cuda(x)
    y = torch.empty((B, N, H, M), dtype=dtype, device=dev)
    ws, pws, nws = _scratch(lib().la_scan_workspace_bytes(0, B, H, G, N, D, M, code), x)
    _check(lib().la_scan_fwd(*ptrs, pS, y.data_ptr(), pws, nws, B, H, G, N, D, M, *ld, code, _stream(None)),
           "la_scan_fwd")
    return y


@_on_device
def scan_bwd(x, dt, A, Bm, Cm, skip, dt_bias, dy, lengths=None):
    """(dx, ddt, dA, dBm, dCm, dskip, ddt_bias) of sum(dy * y) for a zero state before row 0; dskip
    and ddt_bias are None without their parameters."""
    ptrs, ld, (H, G, D, M), code, dtype, dev = _scan_args(x, dt, A, Bm, Cm, skip, dt_bias, lengths, 2)
    B, N = x.shape[:2]
    pg = _take(dy, "dy", x.shape, dtype, dev)
    _need_cuda(x)
    new, h = functools.partial(torch.empty, dtype=dtype, device=dev), (H,)
    d = (new((B, N, H, M)), new((B, N, H)), new(h), new((B, N, G, D)), new((B, N, G, D)), None if skip is None else new(h),
         None if dt_bias is None else new(h))
    ws, pws, nws = _scratch(lib().la_scan_workspace_bytes(1, B, H, G, N, D, M, code), x)
    _check(lib().la_scan_bwd(*ptrs, pg, *[None if t is None else t.data_ptr() for t in d], pws, nws, B, H, G, N, D,
                             M, *ld, code, _stream(None)), "la_scan_bwd")
    return d


@_on_device
def scan_step(x, dt, A, Bm, Cm, skip, dt_bias, S):
    """y [B,H,M] for one row of each stream: x [B,H,M], dt [B,H], Bm and Cm [B,G,D]; S [B,H,D,M]
    (float32) is updated in place."""
    ptrs, ld, (H, G, D, M), code, dtype, dev = _scan_args(x, dt, A, Bm, Cm, skip, dt_bias, None, 1)
    B = x.shape[0]
    pS = _take(S, "S", (B, H, D, M), torch.float32, dev)
    _need_cuda(x)
    y = torch.empty((B, H, M), dtype=dtype, device=dev)
    _check(lib().la_scan_step(*ptrs[:7], pS, y.data_ptr(), B, H, G, D, M, *ld, code, _stream(None)), "la_scan_step")
    return y


def _cross_args(q, k, v, lengths):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v: 4 dimensions")
    B, H, Nq, D = q.shape
    Hk, Nk, M = k.shape[1], k.shape[2], v.shape[3]
    _need_ints(q, k, v)
    code, dtype, dev = _dtype_code(q), q.dtype, q.device
    ptrs = (_take(q, "q", q.shape, dtype, dev), _take(k, "k", (B, Hk, Nk, D), dtype, dev),
            _take(v, "v", (B, Hk, Nk, M), dtype, dev), _take_opt(lengths, "lengths", (B,), torch.int32, dev))
    return ptrs, (B, H, Hk, Nq, Nk, D, M), code, dtype, dev


@_on_device
def cross_fwd(q, k, v, lengths=None):
    """(out, den, S, Z) of the kernelized cross attention of q [B,H,Nq,D] to an encoder's k [B,Hk,Nk,D]
    and v [B,Hk,Nk,M] (Hk divides H); lengths: int32 [B] of valid encoder states.  S [B,Hk,D,M] and
    Z [B,Hk,D] (float32) are all that cross_step needs of the encoder."""
    ptrs, size, code, dtype, dev = _cross_args(q, k, v, lengths)
    B, H, Hk, Nq, Nk, D, M = size
    _need_cuda(q)
    new = functools.partial(torch.empty, dtype=torch.float32, device=dev)
    out, den = torch.empty((B, H, Nq, M), dtype=dtype, device=dev), new((B, H, Nq))
    S, Z = new((B, Hk, D, M)), new((B, Hk, D))
    ws, pws, nws = _scratch(lib().la_cross_workspace_bytes(0, *size, code), q)
    _check(lib().la_cross_fwd(*ptrs, out.data_ptr(), den.data_ptr(), S.data_ptr(), Z.data_ptr(), pws, nws, *size,
                              code, _stream(None)), "la_cross_fwd")
    return out, den, S, Z


@_on_device
def cross_bwd(q, k, v, lengths, out, den, S, Z, dout):
    """(dq, dk, dv) of sum(dout * out); out (not read, may be None), den, S, Z from cross_fwd."""
    ptrs, size, code, dtype, dev = _cross_args(q, k, v, lengths)
    B, H, Hk, Nq, Nk, D, M = size
    f32 = torch.float32
    more = (_take_opt(out, "out", (B, H, Nq, M), dtype, dev), _take(den, "den", (B, H, Nq), f32, dev),
            _take(S, "S", (B, Hk, D, M), f32, dev), _take(Z, "Z", (B, Hk, D), f32, dev),
            _take(dout, "dout", (B, H, Nq, M), dtype, dev))
    _need_cuda(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws, pws, nws = _scratch(lib().la_cross_workspace_bytes(1, *size, code), q)
    _check(lib().la_cross_bwd(*ptrs, *more, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), pws, nws, *size, code,
                              _stream(None)), "la_cross_bwd")
    return dq, dk, dv


@_on_device
def cross_step(q, S, Z):
    """y [B,H,M] for one token q [B,H,D] of each stream, from the kept S [B,Hk,D,M] and Z [B,Hk,D]."""
    if q.dim() != 3 or S.dim() != 4:
        raise ValueError("q: 3 dimensions, S: 4")
    B, H, D = q.shape
    Hk, M = S.shape[1], S.shape[3]
    _need_ints(q, S)
    code, dtype, dev = _dtype_code(q), q.dtype, q.device
    pq = _take(q, "q", q.shape, dtype, dev)
    pS = _take(S, "S", (B, Hk, D, M), torch.float32, dev)
    pZ = _take(Z, "Z", (B, Hk, D), torch.float32, dev)
    _need_cuda(q)
    y = torch.empty((B, H, M), dtype=dtype, device=dev)
    _check(lib().la_cross_step(pq, pS, pZ, y.data_ptr(), B, H, Hk, D, M, code, _stream(None)), "la_cross_step")
    return y


class _Causal(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out, den = causal_fwd(q, k, v)
        ctx.save_for_backward(q, k, v, out, den)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, den = ctx.saved_tensors
        return causal_bwd(q, k, v, out, den, dout.contiguous())


class _NonCausal(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lengths):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out, den, S, Z = noncausal_fwd(q, k, v, lengths)
        ctx.save_for_backward(q, k, v, out, den, S, Z)
        ctx.lengths = lengths
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, den, S, Z = ctx.saved_tensors
        dq, dk, dv = noncausal_bwd(q, k, v, ctx.lengths, out, den, S, Z, dout.contiguous())
        return dq, dk, dv, None


def causal_linear_attention(q, k, v):
    """Causal elu+1 linear attention with the constant-memory backward."""
    return _Causal.apply(q, k, v)


def noncausal_linear_attention(q, k, v, lengths=None):
    """Non-causal elu+1 linear attention (shared S, Z per sequence)."""
    return _NonCausal.apply(q, k, v, lengths)


def _gradient(t):
    """A gradient as the calls need it: autograd hands over views, with any strides and from any address."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _ShortConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, lengths, silu):
        ctx.save_for_backward(x, w, bias, lengths)
        ctx.silu = silu
        return short_conv_fwd(x, w, bias, None, lengths, silu)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, bias, lengths = ctx.saved_tensors
        return *short_conv_bwd(x, w, bias, _gradient(dy), lengths, ctx.silu), None, None


class _Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, Bm, Cm, skip, dt_bias, lengths):
        ctx.save_for_backward(x, dt, A, Bm, Cm, skip, dt_bias, lengths)
        return scan_fwd(x, dt, A, Bm, Cm, skip, dt_bias, None, lengths)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        *inputs, lengths = ctx.saved_tensors
        return *scan_bwd(*inputs, _gradient(dy), lengths), None


class _Cross(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lengths):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        out, den, S, Z = cross_fwd(q, k, v, lengths)
        ctx.save_for_backward(q, k, v, lengths, den, S, Z)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, lengths, den, S, Z = ctx.saved_tensors
        return *cross_bwd(q, k, v, lengths, None, den, S, Z, _gradient(dout)), None


def short_conv(x, w, bias=None, lengths=None, silu=True):
    """short_conv_fwd with its gradients (history zero)."""
    return _ShortConv.apply(x, w, bias, lengths, silu)


def selective_scan(x, dt, A, Bm, Cm, skip=None, dt_bias=None, lengths=None):
    """scan_fwd with its gradients (zero state before row 0; nothing of the forward pass is kept but
    its inputs)."""
    return _Scan.apply(x, dt, A, Bm, Cm, skip, dt_bias, lengths)


def cross_linear_attention(q, k, v, lengths=None):
    """Kernelized cross attention to an encoder's states (cross_fwd) with its gradients."""
    return _Cross.apply(q, k, v, lengths)
