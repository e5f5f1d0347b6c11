"""Binding of the gated feed-forward block and the 4-bit weights
(include/sgemm_f32_ffn.h): argument marshalling only, as in the package.

C-ABI mirrors (same names, same argument order; matrices may be torch tensors
or raw device addresses as ints; they return the C status code):
    sgemm_f32_glu(dtype, act, M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, H, ldh, P, ldp, stream=None)
    sgemm_f32_glu_bwd(dtype, act, M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, P, ldp, dH, lddh, dX, lddx,
                      dWg, lddwg, dWu, lddwu, workspace, workspace_bytes, stream=None)
    sgemm_f32_glu_bwd_ws_size(dtype, M, F, K, num_cus) -> (code, bytes)
    sgemm_f32_w4_quantize(dtype, F, K, group, W, ldw, Q, ldq, S, lds, Z, ldz, stream=None)
    sgemm_f32_w4_dequantize(dtype, F, K, group, Q, ldq, S, lds, Z, ldz, W, ldw, stream=None)
    sgemm_f32_w4(dtype, M, F, K, group, X, ldx, Q, ldq, S, lds, Z, ldz, Y, ldy, stream=None)
    sgemm_f32_w4_glu(dtype, act, M, F, K, group, X, ldx, Qg, Qu, ldq, Sg, Su, lds, Zg, Zu, ldz,
                     H, ldh, stream=None)

Tensor helpers (CUDA tensors of one type -- float32, bfloat16 or float16 -- on
one device, 2-D with unit column stride; any row stride). They check their
arguments, raise SgemmError for a C error code, enqueue on `stream` (default:
the current stream of the tensors' device) and return their outputs; an output
that is not given is allocated, in memory of that stream's own. A call on a stream
that is not the current one waits for nothing there, nor does the current one
wait for the call. No autograd graph is recorded; glu_backward is called
explicitly:
    glu(X, Wg, Wu, act="silu", out=None, preact=None, stream=None)
    glu_backward(dH, X, Wg, Wu, preact, act="silu", dX=None, dWg=None, dWu=None,
                 workspace=None, stream=None)
    w4_quantize(W, group=128, zeros=False, stream=None) -> W4
    w4_dequantize(w, out=None, stream=None)
    w4_matmul(X, w, out=None, stream=None)
    w4_glu(X, wg, wu, act="silu", out=None, stream=None)
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Tuple

from . import SgemmError, _lib, _ptr, _stream

try:
    import torch
except ImportError:   # the C-ABI mirrors need no torch
    torch = None

DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = 0, 1, 2, 3
ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU}

_c, _i, _p, _z = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_m = [_p, _i]   # a matrix and its leading dimension
_SIGNATURES = {
    "sgemm_f32_glu": [_c, _c, _i, _i, _i] + 5 * _m + [_p],
    "sgemm_f32_glu_bwd": [_c, _c, _i, _i, _i] + 8 * _m + [_p, _z, _p],
    "sgemm_f32_glu_bwd_ws_size": [_c, _i, _i, _i, _c, ctypes.POINTER(_z)],
    "sgemm_f32_w4_quantize": [_c, _i, _i, _i] + 4 * _m + [_p],
    "sgemm_f32_w4_dequantize": [_c, _i, _i, _i] + 4 * _m + [_p],
    "sgemm_f32_w4": [_c, _i, _i, _i, _i] + 5 * _m + [_p],
    "sgemm_f32_w4_glu": [_c, _c, _i, _i, _i, _i] + _m + 3 * [_p, _p, _i] + _m + [_p],
}
for _name, _types in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _types
    getattr(_lib, _name).restype = _c


# --------------------------------------------------------------------------
# C-ABI mirrors
# --------------------------------------------------------------------------
def sgemm_f32_glu(dtype, act, M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, H, ldh, P, ldp, stream=None) -> int:
    return _lib.sgemm_f32_glu(dtype, act, M, F, K, _ptr(X), ldx, _ptr(Wg), ldwg, _ptr(Wu), ldwu, _ptr(H),
                              ldh, _ptr(P), ldp, _stream(stream, H, X))


def sgemm_f32_glu_bwd(dtype, act, M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, P, ldp, dH, lddh, dX, lddx, dWg,
                      lddwg, dWu, lddwu, workspace, workspace_bytes, stream=None) -> int:
    return _lib.sgemm_f32_glu_bwd(dtype, act, M, F, K, _ptr(X), ldx, _ptr(Wg), ldwg, _ptr(Wu), ldwu, _ptr(P),
                                  ldp, _ptr(dH), lddh, _ptr(dX), lddx, _ptr(dWg), lddwg, _ptr(dWu), lddwu,
                                  _ptr(workspace), workspace_bytes, _stream(stream, dH, X))


@functools.lru_cache(maxsize=256)
def sgemm_f32_glu_bwd_ws_size(dtype, M, F, K, num_cus) -> Tuple[int, int]:
    b = ctypes.c_size_t(0)
    rc = _lib.sgemm_f32_glu_bwd_ws_size(dtype, M, F, K, num_cus, ctypes.byref(b))
    return int(rc), int(b.value)


def sgemm_f32_w4_quantize(dtype, F, K, group, W, ldw, Q, ldq, S, lds, Z, ldz, stream=None) -> int:
    return _lib.sgemm_f32_w4_quantize(dtype, F, K, group, _ptr(W), ldw, _ptr(Q), ldq, _ptr(S), lds, _ptr(Z),
                                      ldz, _stream(stream, Q, W))


def sgemm_f32_w4_dequantize(dtype, F, K, group, Q, ldq, S, lds, Z, ldz, W, ldw, stream=None) -> int:
    return _lib.sgemm_f32_w4_dequantize(dtype, F, K, group, _ptr(Q), ldq, _ptr(S), lds, _ptr(Z), ldz,
                                        _ptr(W), ldw, _stream(stream, W, Q))


def sgemm_f32_w4(dtype, M, F, K, group, X, ldx, Q, ldq, S, lds, Z, ldz, Y, ldy, stream=None) -> int:
    return _lib.sgemm_f32_w4(dtype, M, F, K, group, _ptr(X), ldx, _ptr(Q), ldq, _ptr(S), lds, _ptr(Z), ldz,
                             _ptr(Y), ldy, _stream(stream, Y, X))


def sgemm_f32_w4_glu(dtype, act, M, F, K, group, X, ldx, Qg, Qu, ldq, Sg, Su, lds, Zg, Zu, ldz, H, ldh,
                     stream=None) -> int:
    return _lib.sgemm_f32_w4_glu(dtype, act, M, F, K, group, _ptr(X), ldx, _ptr(Qg), _ptr(Qu), ldq, _ptr(Sg),
                                 _ptr(Su), lds, _ptr(Zg), _ptr(Zu), ldz, _ptr(H), ldh, _stream(stream, H, X))


# --------------------------------------------------------------------------
# Tensor helpers
# --------------------------------------------------------------------------
class W4(NamedTuple):
    """A weight matrix of `K` inputs in 4 bits: `q` (uint8, rows of at least
    (K + 1) / 2 bytes, the even inputs in the low halves), `scales` and
    `zeros` (None: 8 everywhere), one for each `group` inputs of a row."""
    q: object
    scales: object
    zeros: Optional[object]
    K: int
    group: int


if torch is not None:
    _dtypes = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    # device index -> address of its current stream
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _dtype(t, name: str) -> int:
    d = _dtypes.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return d


def _act(act) -> int:
    a = ACTS.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTS)}")
    return a


def _ld(t, like, dtype, rows: int, cols: int, name: str) -> int:
    """The leading dimension of a rows x cols matrix on `like`'s device."""
    if t.dtype is dtype and t.get_device() == like.get_device() and t.shape == (rows, cols):
        sr, sc = t.stride()
        if sc == 1 or cols == 1:
            if rows == 1:
                return cols or 1
            if rows and sr >= cols > 0:
                return sr
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    sr, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name} must be row-major with unit column stride, got strides {(sr, sc)}")
    if rows <= 1:
        return max(cols, 1)
    if sr < cols:
        raise ValueError(f"the rows of {name} overlap (strides {(sr, sc)})")
    return max(sr, 1)


def _gpu(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return _dtype(t, name)


_entries = {name: getattr(_lib, name) for name in _SIGNATURES}


def _call(like, stream, entry: str, *args) -> None:
    """Calls the C entry point with `like`'s device current."""
    index = like.get_device()
    if _device() == index:
        rc = _entries[entry](*args, _raw_stream(index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(index):
            rc = _entries[entry](*args, _raw_stream(index) if stream is None else _stream(stream))
    if rc != 0:
        raise SgemmError(rc, entry)


def _checked(stream, device):
    """`stream`, a torch stream of the operands' device, an address or None. A
    kernel on another device's stream would run there, on memory that device
    need not reach."""
    if stream is not None and not isinstance(stream, int) and getattr(stream, "device", device) != device:
        raise ValueError(f"the stream is on {stream.device}, the operands are on {device}")
    return stream


def _new(like, rows: int, cols: Optional[int], stream=None, dtype=None, returned: bool = True):
    """A matrix (without `cols` a vector) for a call that works on `stream`, in memory of that stream's own:
    what the current stream has set free may still be read or written by work
    that waits there, which `stream` does not wait for. The caller may use what is
    `returned` on the current stream (once that has waited for the call): its
    memory is not handed on before such use is over."""
    shape = (rows,) if cols is None else (rows, cols)
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=like.device)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if returned:
        t.record_stream(torch.cuda.current_stream(like.device))
    return t


def glu(X, Wg, Wu, act: str = "silu", out=None, preact=None, stream=None):
    """act(X Wg^T) * (X Wu^T). X: (M, K), Wg and Wu: (F, K); returns (M, F).
    `preact`, a float32 (M, 2F) tensor, receives what glu_backward needs."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M, K = X.shape
    F = Wg.shape[0]
    H = _new(X, M, F, stream) if out is None else out
    t = X.dtype
    ldp = 2 * F
    if preact is not None:
        ldp = _ld(preact, X, torch.float32, M, 2 * F, "preact")
    _call(X, stream, "sgemm_f32_glu", d, _act(act), M, F, K, X.data_ptr(), _ld(X, X, t, M, K, "X"),
          Wg.data_ptr(), _ld(Wg, X, t, F, K, "Wg"), Wu.data_ptr(), _ld(Wu, X, t, F, K, "Wu"), H.data_ptr(),
          _ld(H, X, t, M, F, "out"), None if preact is None else preact.data_ptr(), max(ldp, 1))
    return H


def glu_backward(dH, X, Wg, Wu, preact, act: str = "silu", dX=None, dWg=None, dWu=None, workspace=None,
                 stream=None):
    """The gradients (dX, dWg, dWu) of glu() for dH, from the `preact` that it
    filled. Each of the three is written where a tensor is given, allocated
    where it is None, and left out (None in the result) where it is False.
    `workspace`: a CUDA tensor of at least glu_backward_workspace() bytes."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M, K = X.shape
    F = Wg.shape[0]
    t = X.dtype
    got, args = [], []
    for g, rows, name in ((dX, M, "dX"), (dWg, F, "dWg"), (dWu, F, "dWu")):
        if g is False:
            got.append(None)
            args += [None, max(K, 1)]
        else:
            g = _new(X, rows, K, stream) if g is None else g
            got.append(g)
            args += [g.data_ptr(), _ld(g, X, t, rows, K, name)]
    need = glu_backward_workspace(X, F)
    if workspace is None:
        workspace = _new(X, 1, need, stream, torch.uint8, returned=False)
    elif workspace.device != X.device:
        raise ValueError(f"workspace is on {workspace.device}, not on {X.device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _call(X, stream, "sgemm_f32_glu_bwd", d, _act(act), M, F, K, X.data_ptr(), _ld(X, X, t, M, K, "X"),
          Wg.data_ptr(), _ld(Wg, X, t, F, K, "Wg"), Wu.data_ptr(), _ld(Wu, X, t, F, K, "Wu"),
          preact.data_ptr(), _ld(preact, X, torch.float32, M, 2 * F, "preact"), dH.data_ptr(),
          _ld(dH, X, t, M, F, "dH"), *args, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return tuple(got)


_cus = {}


def glu_backward_workspace(X, F: int) -> int:
    """Bytes of workspace glu_backward needs for X (M, K) and F features."""
    d = _gpu(X, "X")
    cus = _cus.get(X.get_device())
    if cus is None:
        cus = _cus[X.get_device()] = torch.cuda.get_device_properties(X.device).multi_processor_count
    rc, need = sgemm_f32_glu_bwd_ws_size(d, X.shape[0], F, X.shape[1], cus)
    if rc != 0:
        raise SgemmError(rc, "sgemm_f32_glu_bwd_ws_size")
    return need


def _groups(K: int, group: int) -> int:
    if group < 1 or (group % 32 and group < K):
        raise ValueError(f"group must be a positive multiple of 32 or at least K = {K}, got {group}")
    return -(-K // group)


def _w4(w: W4, like, name: str):
    """(F, the C arguments) of a 4-bit weight matrix."""
    F, G = w.q.shape[0], _groups(w.K, w.group)
    if w.q.dim() != 2 or w.q.shape[1] != (w.K + 1) // 2:
        raise ValueError(f"{name}.q must have shape (F, {(w.K + 1) // 2}), got {tuple(w.q.shape)}")
    ldq = _ld(w.q, like, torch.uint8, F, (w.K + 1) // 2, f"{name}.q")
    lds = _ld(w.scales, like, like.dtype, F, G, f"{name}.scales")
    ldz = lds if w.zeros is None else _ld(w.zeros, like, like.dtype, F, G, f"{name}.zeros")
    return F, (w.q.data_ptr(), ldq), (w.scales.data_ptr(), lds), (
        None if w.zeros is None else w.zeros.data_ptr(), ldz)


def w4_quantize(W, group: int = 128, zeros: bool = False, stream=None) -> W4:
    """W (F, K) in 4 bits, with zero points where `zeros`."""
    d = _gpu(W, "W")
    stream = _checked(stream, W.device)
    F, K = W.shape
    G = _groups(K, group)
    q = _new(W, F, (K + 1) // 2, stream, torch.uint8)
    s = _new(W, F, G, stream)
    z = _new(W, F, G, stream) if zeros else None
    _call(W, stream, "sgemm_f32_w4_quantize", d, F, K, group, W.data_ptr(), _ld(W, W, W.dtype, F, K, "W"),
          q.data_ptr(), max((K + 1) // 2, 1), s.data_ptr(), max(G, 1), z.data_ptr() if zeros else None, max(G, 1))
    return W4(q, s, z, K, group)


def w4_dequantize(w: W4, out=None, stream=None):
    """The matrix (F, K) that `w` stands for, in the type of its scales."""
    d = _gpu(w.scales, "scales")
    stream = _checked(stream, w.scales.device)
    F, q, s, z = _w4(w, w.scales, "w")
    out = _new(w.scales, F, w.K, stream) if out is None else out
    _call(w.scales, stream, "sgemm_f32_w4_dequantize", d, F, w.K, w.group, *q, *s, *z, out.data_ptr(),
          _ld(out, w.scales, w.scales.dtype, F, w.K, "out"))
    return out


def w4_matmul(X, w: W4, out=None, stream=None):
    """X W^T with W in 4 bits. X: (M, K); returns (M, F). Made for batches of up to
    some 300 rows: longer 16-bit prompts are faster through w4_dequantize and a
    16-bit product of the program's own (the package's dense product, gemm(),
    takes FP32 only)."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M = X.shape[0]
    F, q, s, z = _w4(w, X, "w")
    Y = _new(X, M, F, stream) if out is None else out
    _call(X, stream, "sgemm_f32_w4", d, M, F, w.K, w.group, X.data_ptr(), _ld(X, X, X.dtype, M, w.K, "X"),
          *q, *s, *z, Y.data_ptr(), _ld(Y, X, X.dtype, M, F, "out"))
    return Y


def w4_glu(X, wg: W4, wu: W4, act: str = "silu", out=None, stream=None):
    """act(X Wg^T) * (X Wu^T) with both weights in 4 bits, of the same K,
    group and row strides. Made for batches of up to some 300 rows: longer 16-bit
    prompts are faster through w4_dequantize of both weights and glu()."""
    d = _gpu(X, "X")
    stream = _checked(stream, X.device)
    M = X.shape[0]
    F, qg, sg, zg = _w4(wg, X, "wg")
    Fu, qu, su, zu = _w4(wu, X, "wu")
    if Fu != F or (wg.K, wg.group) != (wu.K, wu.group) or (wg.zeros is None) != (wu.zeros is None):
        raise ValueError("wg and wu must have the same shape and group, and both or neither zero points")
    if qg[1] != qu[1] or sg[1] != su[1] or zg[1] != zu[1]:
        raise ValueError("wg and wu must have the same row strides")
    H = _new(X, M, F, stream) if out is None else out
    _call(X, stream, "sgemm_f32_w4_glu", d, _act(act), M, F, wg.K, wg.group, X.data_ptr(),
          _ld(X, X, X.dtype, M, wg.K, "X"), qg[0], qu[0], qg[1], sg[0], su[0], sg[1], zg[0], zu[0], zg[1],
          H.data_ptr(), _ld(H, X, X.dtype, M, F, "out"))
    return H
