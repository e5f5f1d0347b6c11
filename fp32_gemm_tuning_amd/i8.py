"""Binding of the root-mean-square norm and of matrices in 8 bits
(include/sgemm_f32_i8.h): argument marshalling only, as in ffn.py.

C-ABI mirrors (same names, same argument order; matrices may be torch tensors
or raw device addresses as ints; they return the C status code):
    sgemm_f32_rms_norm(dtype, M, K, eps, X, ldx, R, ldr, W, H, ldh, rstd, Y, ldy, stream=None)
    sgemm_f32_rms_norm_i8(dtype, M, K, eps, X, ldx, R, ldr, W, H, ldh, Q, ldq, S, stream=None)
    sgemm_f32_rms_norm_bwd(dtype, M, K, dY, lddy, W, H, ldh, rstd, dH, lddh, dX, lddx, dW, workspace,
                           workspace_bytes, stream=None)
    sgemm_f32_rms_norm_bwd_ws_size(dtype, M, K) -> (code, bytes)
    sgemm_f32_i8_quantize(dtype, M, K, X, ldx, Q, ldq, S, stream=None)
    sgemm_f32_i8_dequantize(dtype, M, K, Q, ldq, S, X, ldx, stream=None)
    sgemm_f32_i8(dtype, M, F, K, X, ldx, Sx, W, ldw, Sw, Y, ldy, stream=None)
    sgemm_f32_i8_glu(dtype, act, M, F, K, X, ldx, Sx, Wg, ldwg, Sg, Wu, ldwu, Su, H, ldh, stream=None)
and, of include/sgemm_f32_probe.h, the name of the kernel that a product takes (None: none):
    sgemm_f32_i8_kernel(gated, M, F, K, X, ldx, Wg, ldwg, Wu=None, ldwu=1)

Tensor helpers, with ffn.py's rules for tensors, streams, errors and allocated outputs
(norm weights, scales and rstd are 1-D and contiguous):
    rms_norm(X, W, eps=1e-6, residual=None, out=None, total=None, rstd=None, stream=None)
    rms_norm_backward(dY, H, W, rstd, dH=None, dX=None, dW=None, workspace=None, stream=None)
    rms_norm_i8(X, W, eps=1e-6, residual=None, out=None, total=None, stream=None) -> I8
    i8_quantize(X, out=None, stream=None) -> I8
    i8_dequantize(x, dtype=torch.float32, out=None, stream=None)
    i8_matmul(x, w, dtype=torch.float32, out=None, stream=None)
    i8_glu(x, wg, wu, act="silu", dtype=torch.float32, out=None, stream=None)
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Tuple

from . import SgemmError, _lib, _ptr, _stream
from .ffn import _act, _c, _call, _checked, _entries, _gpu, _i, _ld, _m, _new, _p, _z

try:
    import torch

    from .ffn import _dtypes
except ImportError:   # the C-ABI mirrors need no torch
    torch = None

_f = ctypes.c_float
_SIGNATURES = {
    "sgemm_f32_rms_norm": [_c, _i, _i, _f] + 2 * _m + [_p] + _m + [_p] + _m + [_p],
    "sgemm_f32_rms_norm_i8": [_c, _i, _i, _f] + 2 * _m + [_p] + 2 * _m + [_p, _p],
    "sgemm_f32_rms_norm_bwd": [_c, _i, _i] + _m + [_p] + _m + [_p] + 2 * _m + [_p, _p, _z, _p],
    "sgemm_f32_rms_norm_bwd_ws_size": [_c, _i, _i, ctypes.POINTER(_z)],
    "sgemm_f32_i8_quantize": [_c, _i, _i] + 2 * _m + [_p, _p],
    "sgemm_f32_i8_dequantize": [_c, _i, _i] + _m + [_p] + _m + [_p],
    "sgemm_f32_i8": [_c, _i, _i, _i] + 2 * (_m + [_p]) + _m + [_p],
    "sgemm_f32_i8_glu": [_c, _c, _i, _i, _i] + 3 * (_m + [_p]) + _m + [_p],
}
for _name, _types in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _types
    getattr(_lib, _name).restype = _c
    _entries[_name] = getattr(_lib, _name)


_lib.sgemm_f32_i8_kernel.argtypes = [_c, _i, _i, _i] + 3 * _m
_lib.sgemm_f32_i8_kernel.restype = ctypes.c_char_p


# --------------------------------------------------------------------------
# C-ABI mirrors
# --------------------------------------------------------------------------
def sgemm_f32_rms_norm(dtype, M, K, eps, X, ldx, R, ldr, W, H, ldh, rstd, Y, ldy, stream=None) -> int:
    return _lib.sgemm_f32_rms_norm(dtype, M, K, eps, _ptr(X), ldx, _ptr(R), ldr, _ptr(W), _ptr(H), ldh,
                                   _ptr(rstd), _ptr(Y), ldy, _stream(stream, Y, X))


def sgemm_f32_rms_norm_i8(dtype, M, K, eps, X, ldx, R, ldr, W, H, ldh, Q, ldq, S, stream=None) -> int:
    return _lib.sgemm_f32_rms_norm_i8(dtype, M, K, eps, _ptr(X), ldx, _ptr(R), ldr, _ptr(W), _ptr(H), ldh,
                                      _ptr(Q), ldq, _ptr(S), _stream(stream, Q, X))


def sgemm_f32_rms_norm_bwd(dtype, M, K, dY, lddy, W, H, ldh, rstd, dH, lddh, dX, lddx, dW, workspace,
                           workspace_bytes, stream=None) -> int:
    return _lib.sgemm_f32_rms_norm_bwd(dtype, M, K, _ptr(dY), lddy, _ptr(W), _ptr(H), ldh, _ptr(rstd), _ptr(dH),
                                       lddh, _ptr(dX), lddx, _ptr(dW), _ptr(workspace), workspace_bytes,
                                       _stream(stream, dY, H))


@functools.lru_cache(maxsize=256)
def sgemm_f32_rms_norm_bwd_ws_size(dtype, M, K) -> Tuple[int, int]:
    b = ctypes.c_size_t(0)
    rc = _lib.sgemm_f32_rms_norm_bwd_ws_size(dtype, M, K, ctypes.byref(b))
    return int(rc), int(b.value)


def sgemm_f32_i8_quantize(dtype, M, K, X, ldx, Q, ldq, S, stream=None) -> int:
    return _lib.sgemm_f32_i8_quantize(dtype, M, K, _ptr(X), ldx, _ptr(Q), ldq, _ptr(S), _stream(stream, Q, X))


def sgemm_f32_i8_dequantize(dtype, M, K, Q, ldq, S, X, ldx, stream=None) -> int:
    return _lib.sgemm_f32_i8_dequantize(dtype, M, K, _ptr(Q), ldq, _ptr(S), _ptr(X), ldx, _stream(stream, X, Q))


def sgemm_f32_i8(dtype, M, F, K, X, ldx, Sx, W, ldw, Sw, Y, ldy, stream=None) -> int:
    return _lib.sgemm_f32_i8(dtype, M, F, K, _ptr(X), ldx, _ptr(Sx), _ptr(W), ldw, _ptr(Sw), _ptr(Y), ldy,
                             _stream(stream, Y, X))


def sgemm_f32_i8_glu(dtype, act, M, F, K, X, ldx, Sx, Wg, ldwg, Sg, Wu, ldwu, Su, H, ldh, stream=None) -> int:
    return _lib.sgemm_f32_i8_glu(dtype, act, M, F, K, _ptr(X), ldx, _ptr(Sx), _ptr(Wg), ldwg, _ptr(Sg), _ptr(Wu),
                                 ldwu, _ptr(Su), _ptr(H), ldh, _stream(stream, H, X))


def sgemm_f32_i8_kernel(gated, M, F, K, X, ldx, Wg, ldwg, Wu=None, ldwu=1):
    name = _lib.sgemm_f32_i8_kernel(int(gated), M, F, K, _ptr(X), ldx, _ptr(Wg), ldwg, _ptr(Wu), ldwu)
    return None if name is None else name.decode()


# --------------------------------------------------------------------------
# Tensor helpers
# --------------------------------------------------------------------------
class I8(NamedTuple):
    """A matrix in 8 bits: `q` (int8, any row stride) and `scales` (float32, one
    for each row)."""
    q: object
    scales: object


def _vec(t, like, dtype, n: int, name: str) -> int:
    """The address of a contiguous vector of n elements on `like`'s device."""
    if t.dtype is dtype and t.shape == (n,) and t.get_device() == like.get_device() and t.stride(0) == 1:
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,):
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous, got stride {t.stride(0)}")
    return t.data_ptr()


def _i8(x, like, name: str):
    """(rows, K, the C arguments) of a matrix in 8 bits."""
    q = x.q
    if q.dim() != 2:
        raise ValueError(f"{name}.q must be 2-D, got shape {tuple(q.shape)}")
    if not q.is_cuda:
        raise ValueError(f"{name}.q must be a GPU tensor")
    rows, K = q.shape
    return rows, K, (q.data_ptr(), _ld(q, like, torch.int8, rows, K, f"{name}.q"),
                     _vec(x.scales, like, torch.float32, rows, f"{name}.scales"))


def _type(dtype, out) -> int:
    """The C dtype of an output: of `out` where it is given."""
    if out is not None:
        dtype = out.dtype
    d = _dtypes.get(dtype)
    if d is None:
        raise TypeError(f"{'out' if out is not None else 'dtype'} must be float32, bfloat16 or float16, got {dtype}")
    return d


def _new_i8(like, M: int, K: int, out, stream) -> I8:
    if out is not None:
        return out
    return I8(_new(like, M, K, stream, torch.int8), _new(like, M, None, stream, torch.float32))


def _or_null(t, like, dtype, rows: int, cols: int, name: str):
    """(address, leading dimension) of a matrix that may be None."""
    return (None, 1) if t is None else (t.data_ptr(), _ld(t, like, dtype, rows, cols, name))


def rms_norm(X, W, eps: float = 1e-6, residual=None, out=None, total=None, rstd=None, stream=None):
    """H rstd W, rstd = 1 / sqrt(mean(H^2) + eps) row by row, of H = X + residual
    (X where there is none). X: (M, K), W: (K,); returns (M, K). `total`, (M, K),
    receives H (it may be X or residual), `rstd`, a float32 (M,) tensor, the
    reciprocal roots: with them rms_norm_backward gives the gradients."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M, K = X.shape
    t = X.dtype
    Y = _new(X, M, K, stream) if out is None else out
    _call(X, stream, "sgemm_f32_rms_norm", d, M, K, eps, X.data_ptr(), _ld(X, X, t, M, K, "X"),
          *_or_null(residual, X, t, M, K, "residual"), _vec(W, X, t, K, "W"), *_or_null(total, X, t, M, K, "total"),
          None if rstd is None else _vec(rstd, X, torch.float32, M, "rstd"), Y.data_ptr(),
          _ld(Y, X, t, M, K, "out"))
    return Y


def rms_norm_backward(dY, H, W, rstd, dH=None, dX=None, dW=None, workspace=None, stream=None):
    """The gradients (dX, dW) of rms_norm() for dY, from its `total` (X where there was
    no residual) and `rstd`; dX is the residual's gradient too. `dH`: the gradient that
    reaches H otherwise (of the residual stream behind the norm), added to dX. Each of the two is
    written where a tensor is given (dX may be dH or dY), allocated where it is None, and
    left out (None in the result) where it is False. `workspace`: a CUDA tensor of at least
    rms_norm_backward_workspace() bytes (any, where dW is left out)."""
    d = _gpu(H, "H")
    stream = _checked(stream, H.device)
    M, K = H.shape
    t = H.dtype
    if dX is None:
        dX = _new(H, M, K, stream)
    if dW is None:
        dW = _new(H, K, None, stream)
    if workspace is None:
        need = 0 if dW is False else rms_norm_backward_workspace(H)
        workspace = _new(H, need, None, stream, torch.uint8, returned=False)
    elif workspace.device != H.device:
        raise ValueError(f"workspace is on {workspace.device}, not on {H.device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _call(H, stream, "sgemm_f32_rms_norm_bwd", d, M, K, dY.data_ptr(), _ld(dY, H, t, M, K, "dY"),
          _vec(W, H, t, K, "W"), H.data_ptr(), _ld(H, H, t, M, K, "H"), _vec(rstd, H, torch.float32, M, "rstd"),
          *_or_null(dH, H, t, M, K, "dH"), *_or_null(None if dX is False else dX, H, t, M, K, "dX"),
          None if dW is False else _vec(dW, H, t, K, "dW"), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return None if dX is False else dX, None if dW is False else dW


def rms_norm_backward_workspace(H) -> int:
    """Bytes of workspace rms_norm_backward needs for H (M, K)."""
    d = _gpu(H, "H")
    rc, need = sgemm_f32_rms_norm_bwd_ws_size(d, H.shape[0], H.shape[1])
    if rc != 0:
        raise SgemmError(rc, "sgemm_f32_rms_norm_bwd_ws_size")
    return need


def rms_norm_i8(X, W, eps: float = 1e-6, residual=None, out=None, total=None, stream=None) -> I8:
    """rms_norm() with its result in 8 bits, (M, K) with a scale for each row, for
    i8_matmul and i8_glu. `out`: an I8 to be written."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M, K = X.shape
    t = X.dtype
    y = _new_i8(X, M, K, out, stream)
    _call(X, stream, "sgemm_f32_rms_norm_i8", d, M, K, eps, X.data_ptr(), _ld(X, X, t, M, K, "X"),
          *_or_null(residual, X, t, M, K, "residual"), _vec(W, X, t, K, "W"), *_or_null(total, X, t, M, K, "total"),
          y.q.data_ptr(), _ld(y.q, X, torch.int8, M, K, "out.q"), _vec(y.scales, X, torch.float32, M, "out.scales"))
    return y


def i8_quantize(X, out=None, stream=None) -> I8:
    """X (M, K) in 8 bits with a scale for each row: activations by token, or a
    weight (F, K) by output feature. `out`: an I8 to be written."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M, K = X.shape
    y = _new_i8(X, M, K, out, stream)
    _call(X, stream, "sgemm_f32_i8_quantize", d, M, K, X.data_ptr(), _ld(X, X, X.dtype, M, K, "X"),
          y.q.data_ptr(), _ld(y.q, X, torch.int8, M, K, "out.q"), _vec(y.scales, X, torch.float32, M, "out.scales"))
    return y


def i8_dequantize(x: I8, dtype=None, out=None, stream=None):
    """The matrix (M, K) that `x` stands for, in `dtype` (float32) or the type of `out`."""
    M, K, (q, ldq, s) = _i8(x, x.q, "x")
    dtype = (torch.float32 if dtype is None else dtype) if out is None else out.dtype
    d = _type(dtype, out)
    stream = _checked(stream, x.q.device)
    out = _new(x.q, M, K, stream, dtype) if out is None else out
    _call(x.q, stream, "sgemm_f32_i8_dequantize", d, M, K, q, ldq, s, out.data_ptr(),
          _ld(out, x.q, dtype, M, K, "out"))
    return out


def i8_matmul(x: I8, w: I8, dtype=None, out=None, stream=None):
    """x w^T of matrices in 8 bits. x: (M, K), w: (F, K); returns (M, F) in
    `dtype` (float32) or the type of `out`."""
    M, K, xs = _i8(x, x.q, "x")
    F = w.q.shape[0]
    if w.q.shape[-1] != K:
        raise ValueError(f"w.q must have shape (F, {K}), got {tuple(w.q.shape)}")
    _, _, ws = _i8(w, x.q, "w")
    dtype = (torch.float32 if dtype is None else dtype) if out is None else out.dtype
    d = _type(dtype, out)
    stream = _checked(stream, x.q.device)
    Y = _new(x.q, M, F, stream, dtype) if out is None else out
    _call(x.q, stream, "sgemm_f32_i8", d, M, F, K, *xs, *ws, Y.data_ptr(), _ld(Y, x.q, dtype, M, F, "out"))
    return Y


def i8_glu(x: I8, wg: I8, wu: I8, act: str = "silu", dtype=None, out=None, stream=None):
    """act(x wg^T) * (x wu^T) of matrices in 8 bits. x: (M, K), wg and wu: (F, K);
    returns (M, F) in `dtype` (float32) or the type of `out`."""
    M, K, xs = _i8(x, x.q, "x")
    F = wg.q.shape[0]
    for w, name in ((wg, "wg"), (wu, "wu")):
        if w.q.shape != (F, K):
            raise ValueError(f"{name}.q must have shape ({F}, {K}), got {tuple(w.q.shape)}")
    dtype = (torch.float32 if dtype is None else dtype) if out is None else out.dtype
    d = _type(dtype, out)
    stream = _checked(stream, x.q.device)
    H = _new(x.q, M, F, stream, dtype) if out is None else out
    _call(x.q, stream, "sgemm_f32_i8_glu", d, _act(act), M, F, K, *xs, *_i8(wg, x.q, "wg")[2],
          *_i8(wu, x.q, "wu")[2], H.data_ptr(), _ld(H, x.q, dtype, M, F, "out"))
    return H
