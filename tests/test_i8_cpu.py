"""Host-side checks of the norm's and the 8-bit entry points, without a GPU:
every function of the header is exported, and each bad argument is refused with
its own code before anything is launched (fake, aligned addresses; only their
alignment is looked at)."""
import ctypes
import inspect
import os
import re

import pytest

torch = pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "sgemm_f32_i8.h")
P = 1 << 20


def test_every_declared_function_is_exported():
    names = re.findall(r"SGEMM_F32_API\s+[^;]*?\b(sgemm_f32\w*)\s*\(", open(HEADER).read())
    assert len(names) == 8
    lib = ctypes.CDLL(sg.LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and hasattr(sg, n), n


@pytest.mark.parametrize("code", range(-46, -37))
def test_each_code_has_a_text(code):
    s = sg.sgemm_f32_strerror(code)
    assert len(s) > 3 and s != "unknown error"


NORM = dict(dtype=0, M=4, K=8, eps=1e-6, X=P, ldx=8, R=P, ldr=8, W=P, H=P, ldh=8, rstd=P, Y=P, ldy=8)
NORM_I8 = dict(dtype=0, M=4, K=8, eps=1e-6, X=P, ldx=8, R=P, ldr=8, W=P, H=P, ldh=8, Q=P, ldq=8, S=P)
BWD = dict(dtype=0, M=4, K=8, dY=P, lddy=8, W=P, H=P, ldh=8, rstd=P, dH=P, lddh=8, dX=P, lddx=8, dW=P, workspace=P,
           workspace_bytes=1 << 30)
QUANT = dict(dtype=0, M=4, K=8, X=P, ldx=8, Q=P, ldq=8, S=P)
DEQUANT = dict(dtype=0, M=4, K=8, Q=P, ldq=8, S=P, X=P, ldx=8)
I8 = dict(dtype=0, M=4, F=6, K=8, X=P, ldx=8, Sx=P, W=P, ldw=8, Sw=P, Y=P, ldy=6)
I8_GLU = dict(dtype=0, act=0, M=4, F=6, K=8, X=P, ldx=8, Sx=P, Wg=P, ldwg=8, Sg=P, Wu=P, ldwu=8, Su=P, H=P, ldh=6)

INPUTS = [("dtype", 3, -17), ("dtype", -1, -17), ("M", -1, -1), ("K", -1, -3), ("eps", -1e-6, -40),
          ("eps", float("inf"), -40), ("eps", float("nan"), -40), ("X", 0, -5), ("X", P + 2, -5), ("ldx", 7, -6),
          ("R", P + 1, -38), ("ldr", 7, -39), ("W", 0, -7), ("W", P + 2, -7), ("H", P + 2, -41), ("ldh", 7, -42)]
BAD = [
    (sg.sgemm_f32_rms_norm, NORM, INPUTS + [("rstd", P + 2, -43), ("Y", 0, -10), ("Y", P + 1, -10), ("ldy", 7, -11)]),
    (sg.sgemm_f32_rms_norm_i8, NORM_I8, INPUTS + [("Q", 0, -7), ("ldq", 7, -8), ("S", 0, -32), ("S", P + 2, -32)]),
    (sg.sgemm_f32_rms_norm_bwd, BWD, [
        ("dtype", 3, -17), ("M", -1, -1), ("K", -1, -3), ("dY", 0, -45), ("dY", P + 2, -45), ("lddy", 7, -46),
        ("W", 0, -7), ("H", 0, -41), ("ldh", 7, -42), ("rstd", 0, -43), ("rstd", P + 2, -43), ("dH", P + 1, -23),
        ("lddh", 7, -24), ("dX", P + 2, -25), ("lddx", 7, -26), ("dW", P + 2, -27), ("workspace", 0, -16),
        ("workspace", P + 8, -16), ("workspace_bytes", 8, sg.ERR_WORKSPACE)]),
    (sg.sgemm_f32_i8_quantize, QUANT, [
        ("dtype", 3, -17), ("M", -1, -1), ("K", -1, -3), ("X", 0, -5), ("X", P + 2, -5), ("ldx", 7, -6), ("Q", 0, -7),
        ("ldq", 7, -8), ("S", 0, -32), ("S", P + 1, -32)]),
    (sg.sgemm_f32_i8_dequantize, DEQUANT, [
        ("dtype", 3, -17), ("M", -1, -1), ("K", -1, -3), ("Q", 0, -7), ("ldq", 7, -8), ("S", 0, -32), ("X", 0, -10),
        ("X", P + 2, -10), ("ldx", 7, -11)]),
    (sg.sgemm_f32_i8, I8, [
        ("dtype", 3, -17), ("M", -1, -1), ("F", -1, -2), ("K", -1, -3), ("X", 0, -5), ("ldx", 7, -6), ("Sx", 0, -44),
        ("Sx", P + 2, -44), ("W", 0, -7), ("ldw", 7, -8), ("Sw", 0, -32), ("Sw", P + 1, -32), ("Y", 0, -10),
        ("Y", P + 2, -10), ("ldy", 5, -11)]),
    (sg.sgemm_f32_i8_glu, I8_GLU, [
        ("dtype", 3, -17), ("act", 4, -18), ("act", -1, -18), ("M", -1, -1), ("F", -1, -2), ("K", -1, -3),
        ("X", 0, -5), ("ldx", 7, -6), ("Sx", 0, -44), ("Wg", 0, -7), ("ldwg", 7, -8), ("Sg", 0, -32), ("Wu", 0, -19),
        ("ldwu", 7, -20), ("Su", 0, -36), ("Su", P + 2, -36), ("H", 0, -10), ("ldh", 5, -11)]),
]


def _names(v):
    return getattr(v, "__name__", None) or (None if isinstance(v, dict) and len(v) > 4 else str(v))


@pytest.mark.parametrize("entry,good,name,value,code", [(e, g, *b) for e, g, bad in BAD for b in bad], ids=_names)
def test_bad_arguments(entry, good, name, value, code):
    assert entry(*dict(good, **{name: value}).values(), stream=0) == code


@pytest.mark.parametrize("entry,good,empty", [
    (sg.sgemm_f32_rms_norm, NORM, dict(M=0)), (sg.sgemm_f32_rms_norm, NORM, dict(K=0, rstd=0)),
    (sg.sgemm_f32_rms_norm_i8, NORM_I8, dict(M=0)), (sg.sgemm_f32_rms_norm_bwd, BWD, dict(K=0)),
    (sg.sgemm_f32_rms_norm_bwd, BWD, dict(dX=0, dW=0)), (sg.sgemm_f32_rms_norm_bwd, BWD, dict(M=0, dW=0)),
    (sg.sgemm_f32_i8_quantize, QUANT, dict(M=0)), (sg.sgemm_f32_i8_dequantize, DEQUANT, dict(M=0)),
    (sg.sgemm_f32_i8_dequantize, DEQUANT, dict(K=0)), (sg.sgemm_f32_i8, I8, dict(M=0)),
    (sg.sgemm_f32_i8, I8, dict(F=0)), (sg.sgemm_f32_i8_glu, I8_GLU, dict(M=0)),
    (sg.sgemm_f32_i8_glu, I8_GLU, dict(F=0))], ids=_names)
def test_empty_outputs_touch_nothing(entry, good, empty):
    # null pointers everywhere: nothing would be read or written
    args = {k: 0 if v == P and k != "workspace" else v for k, v in good.items()}
    assert entry(*dict(args, **empty).values(), stream=0) == 0


@pytest.mark.parametrize("entry,good", [(e, g) for e, g, _ in BAD], ids=_names)
def test_sizes_beyond_the_index_range(entry, good):
    big = 1 << 40
    args = {k: big if k.startswith("ld") else v for k, v in good.items()}
    for name in ("M", "F", "K"):
        if name in args:
            assert entry(*dict(args, **{name: (1 << 30) + 1}).values(), stream=0) == sg.ERR_TOO_LARGE


@pytest.mark.parametrize("entry,good", [(sg.sgemm_f32_i8, I8), (sg.sgemm_f32_i8_glu, I8_GLU)], ids=_names)
def test_sums_beyond_32_bits_are_refused(entry, good):
    args = {k: 1 << 20 if k.startswith("ld") else v for k, v in good.items()}
    assert 131071 * 128 * 128 < 2 ** 31 <= 131072 * 128 * 128
    assert entry(*dict(args, K=131072).values(), stream=0) == sg.ERR_TOO_LARGE


def test_workspace_size():
    for dtype in range(3):
        rc, n = sg.sgemm_f32_rms_norm_bwd_ws_size(dtype, 100, 65)
        assert rc == 0 and n >= 65 * 4
        assert sg.sgemm_f32_rms_norm_bwd_ws_size(dtype, 0, 65) == (0, 0)
        assert sg.sgemm_f32_rms_norm_bwd_ws_size(dtype, 65, 0) == (0, 0)
    assert sg.sgemm_f32_rms_norm_bwd_ws_size(3, 1, 1)[0] == -17
    assert sg.sgemm_f32_rms_norm_bwd_ws_size(0, -1, 1)[0] == -1
    assert sg.sgemm_f32_rms_norm_bwd_ws_size(0, 1, -1)[0] == -3
    assert sg.sgemm_f32_rms_norm_bwd_ws_size(0, 1, 1 << 31)[0] == sg.ERR_TOO_LARGE
    assert sg.i8._lib.sgemm_f32_rms_norm_bwd_ws_size(0, 1, 1, None) == -12
    need = sg.sgemm_f32_rms_norm_bwd_ws_size(1, 4, 8)[1]
    assert sg.sgemm_f32_rms_norm_bwd(*dict(BWD, dtype=1, workspace_bytes=need - 1).values(),
                                     stream=0) == sg.ERR_WORKSPACE
    assert sg.sgemm_f32_rms_norm_bwd(*dict(BWD, workspace=0, workspace_bytes=0).values(),
                                     stream=0) == sg.ERR_WORKSPACE


def test_helpers_refuse_what_they_cannot_pass():
    from fp32_gemm_tuning_amd.i8 import _i8, _type, _vec
    x, q, s = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: sg.rms_norm(x, s), lambda: sg.rms_norm_i8(x, s), lambda: sg.i8_quantize(x),
                 lambda: sg.rms_norm_backward(x, x, s, s), lambda: sg.i8_dequantize(sg.I8(q, s)),
                 lambda: sg.i8_matmul(sg.I8(q, s), sg.I8(q, s)),
                 lambda: sg.i8_glu(sg.I8(q, s), sg.I8(q, s), sg.I8(q, s))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(ValueError, match="2-D"):
        sg.rms_norm(x[0], s)
    with pytest.raises(ValueError, match="2-D"):
        _i8(sg.I8(q[0], s), q, "x")
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sg.rms_norm(GpuTensor(4, 64, dtype=torch.float64), V)
    with pytest.raises(TypeError, match="dtype must be"):
        _type(torch.int8, None)
    with pytest.raises(TypeError, match="out must be"):
        _type(None, q)
    with pytest.raises(TypeError, match="W must be"):
        _vec(s, x, torch.bfloat16, 4, "W")
    with pytest.raises(ValueError, match="shape"):
        _vec(s, x, torch.float32, 8, "W")
    with pytest.raises(ValueError, match="shape"):
        _vec(x, x, torch.float32, 4, "W")
    with pytest.raises(ValueError, match="contiguous"):
        _vec(torch.zeros(8)[::2], x, torch.float32, 4, "W")
    assert _vec(torch.zeros(8)[::8], x, torch.float32, 1, "W")


def test_nothing_is_allocated_another_way():
    source = inspect.getsource(sg.i8)
    assert not re.search(r"torch\.(empty|zeros|ones|full)\w*\(", source) and "new_empty(" not in source


class GpuTensor:
    """What the helpers look at before they look at a stream."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.device, self.dtype = shape, torch.device("cuda:0"), dtype

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        s = (self.shape[1], 1) if self.dim() == 2 else (1,)
        return s if i is None else s[i]

    def get_device(self):
        return 0

    def data_ptr(self):
        return P


class Elsewhere:
    device = torch.device("cuda:1")
    cuda_stream = 4096


X, V = GpuTensor(4, 64), GpuTensor(64)
A = sg.I8(GpuTensor(4, 64, dtype=torch.int8), GpuTensor(4, dtype=torch.float32))


@pytest.mark.parametrize("call", [
    lambda s: sg.rms_norm(X, V, stream=s), lambda s: sg.rms_norm_i8(X, V, stream=s),
    lambda s: sg.rms_norm_backward(X, X, V, V, stream=s), lambda s: sg.i8_quantize(X, stream=s),
    lambda s: sg.i8_dequantize(A, stream=s), lambda s: sg.i8_matmul(A, A, stream=s),
    lambda s: sg.i8_glu(A, A, A, stream=s)],
    ids=["rms_norm", "rms_norm_i8", "rms_norm_backward", "i8_quantize", "i8_dequantize", "i8_matmul", "i8_glu"])
def test_another_devices_stream_is_refused(call):
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(Elsewhere())


@pytest.mark.parametrize("call,match", [
    (lambda: sg.i8_matmul(A, sg.I8(GpuTensor(5, 63, dtype=torch.int8), GpuTensor(5, dtype=torch.float32))), "w.q"),
    (lambda: sg.i8_glu(A, A, sg.I8(GpuTensor(5, 64, dtype=torch.int8), GpuTensor(5, dtype=torch.float32))), "wu.q"),
    (lambda: sg.i8_matmul(sg.I8(A.q, GpuTensor(5, dtype=torch.float32)), A), "x.scales"),
    (lambda: sg.i8_matmul(A, sg.I8(A.q, GpuTensor(4, dtype=torch.bfloat16))), "w.scales")],
    ids=["K", "F", "scales", "type"])
def test_matrices_that_do_not_fit_each_other(call, match):
    with pytest.raises((ValueError, TypeError), match=match):
        call()
