"""Host-side checks of the feed-forward entry points, without a GPU: every
function of the header is exported, and each bad argument is refused with its
own code before anything is launched (fake, aligned addresses; only their
alignment is looked at)."""
import ctypes
import os
import re

import pytest

torch = pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "sgemm_f32_ffn.h")
P = 1 << 20


def test_every_declared_function_is_exported():
    names = re.findall(r"SGEMM_F32_API\s+[^;]*?\b(sgemm_f32\w*)\s*\(", open(HEADER).read())
    assert len(names) == 7
    lib = ctypes.CDLL(sg.LIB_PATH)
    for n in names:
        assert hasattr(lib, n) and hasattr(sg, n), n


def test_enums_match_the_binding():
    enum = {m.group(1): int(m.group(2))
            for m in re.finditer(r"SGEMM_F32_((?:DTYPE|ACT)_\w+)\s*=\s*(\d+)", open(HEADER).read())}
    from fp32_gemm_tuning_amd import ffn
    assert enum == {k: getattr(ffn, k) for k in dir(ffn) if re.match(r"(DTYPE|ACT)_", k)}
    assert {"ACT_" + k.upper(): v for k, v in sg.ACTS.items()} == {k: v for k, v in enum.items() if k[0] == "A"}


@pytest.mark.parametrize("code", [-17 - i for i in range(21)] + [-16, -104])
def test_each_code_has_a_text(code):
    s = sg.sgemm_f32_strerror(code)
    assert len(s) > 3 and s != "unknown error"


GLU = dict(dtype=0, act=0, M=4, F=6, K=8, X=P, ldx=8, Wg=P, ldwg=8, Wu=P, ldwu=8, H=P, ldh=6, P=P, ldp=12)
BWD = dict(dtype=0, act=0, M=4, F=6, K=8, X=P, ldx=8, Wg=P, ldwg=8, Wu=P, ldwu=8, P=P, ldp=12, dH=P, lddh=6,
           dX=P, lddx=8, dWg=P, lddwg=8, dWu=P, lddwu=8, workspace=P, workspace_bytes=1 << 30)
W4 = dict(dtype=0, M=4, F=6, K=65, group=32, X=P, ldx=65, Q=P, ldq=33, S=P, lds=3, Z=P, ldz=3, Y=P, ldy=6)
W4_GLU = dict(dtype=0, act=0, M=4, F=6, K=65, group=32, X=P, ldx=65, Qg=P, Qu=P, ldq=33, Sg=P, Su=P, lds=3,
              Zg=P, Zu=P, ldz=3, H=P, ldh=6)
QUANT = dict(dtype=0, F=6, K=65, group=32, W=P, ldw=65, Q=P, ldq=33, S=P, lds=3, Z=P, ldz=3)
DEQUANT = dict(dtype=0, F=6, K=65, group=32, Q=P, ldq=33, S=P, lds=3, Z=P, ldz=3, W=P, ldw=65)

BAD = [
    (sg.sgemm_f32_glu, GLU, [
        ("dtype", 3, -17), ("dtype", -1, -17), ("act", 4, -18), ("act", -1, -18), ("M", -1, -1), ("F", -1, -2),
        ("K", -1, -3), ("X", 0, -5), ("X", P + 2, -5), ("ldx", 7, -6), ("Wg", 0, -7), ("ldwg", 7, -8),
        ("Wu", P + 1, -19), ("ldwu", 0, -20), ("P", P + 2, -21), ("ldp", 11, -22), ("H", 0, -10), ("ldh", 5, -11)]),
    (sg.sgemm_f32_glu_bwd, BWD, [
        ("dtype", 3, -17), ("act", 4, -18), ("M", -1, -1), ("F", -1, -2), ("K", -1, -3), ("X", 0, -5),
        ("ldx", 7, -6), ("Wg", 0, -7), ("ldwg", 7, -8), ("Wu", 0, -19), ("ldwu", 7, -20), ("P", 0, -21),
        ("ldp", 11, -22), ("dH", 0, -23), ("lddh", 5, -24), ("dX", P + 1, -25), ("lddx", 7, -26),
        ("dWg", P + 2, -27), ("lddwg", 7, -28), ("dWu", P + 3, -29), ("lddwu", 7, -30), ("workspace", 0, -16),
        ("workspace", P + 8, -16)]),
    (sg.sgemm_f32_w4, W4, [
        ("dtype", 3, -17), ("M", -1, -1), ("F", -1, -2), ("K", -1, -3), ("group", 0, -31), ("group", -32, -31),
        ("group", 48, -31), ("X", 0, -5), ("ldx", 64, -6), ("Q", 0, -7), ("ldq", 32, -8), ("S", 0, -32),
        ("S", P + 2, -32), ("lds", 2, -33), ("Z", P + 1, -34), ("ldz", 2, -35), ("Y", 0, -10), ("ldy", 5, -11)]),
    (sg.sgemm_f32_w4_glu, W4_GLU, [
        ("dtype", 3, -17), ("act", 4, -18), ("M", -1, -1), ("F", -1, -2), ("K", -1, -3), ("group", 1, -31),
        ("X", 0, -5), ("ldx", 64, -6), ("Qg", 0, -7), ("Qu", 0, -19), ("ldq", 32, -8), ("Sg", 0, -32),
        ("Su", 0, -36), ("lds", 2, -33), ("Zg", P + 1, -34), ("Zg", 0, -37), ("Zu", 0, -37), ("Zu", P + 1, -37),
        ("ldz", 2, -35), ("H", 0, -10), ("ldh", 5, -11)]),
    (sg.sgemm_f32_w4_quantize, QUANT, [
        ("dtype", 3, -17), ("F", -1, -2), ("K", -1, -3), ("group", 33, -31), ("W", 0, -5), ("ldw", 64, -6),
        ("Q", 0, -7), ("ldq", 32, -8), ("S", 0, -32), ("lds", 2, -33), ("Z", P + 2, -34), ("ldz", 2, -35)]),
    (sg.sgemm_f32_w4_dequantize, DEQUANT, [
        ("dtype", 3, -17), ("F", -1, -2), ("K", -1, -3), ("group", 33, -31), ("Q", 0, -7), ("ldq", 32, -8),
        ("S", 0, -32), ("lds", 2, -33), ("Z", P + 2, -34), ("ldz", 2, -35), ("W", 0, -10), ("ldw", 64, -11)]),
]


@pytest.mark.parametrize("entry,good,name,value,code",
                         [(e, g, *b) for e, g, bad in BAD for b in bad],
                         ids=lambda v: getattr(v, "__name__", None) or (None if isinstance(v, dict) else str(v)))
def test_bad_arguments(entry, good, name, value, code):
    assert entry(*dict(good, **{name: value}).values(), stream=0) == code


@pytest.mark.parametrize("entry,good,empty", [
    (sg.sgemm_f32_glu, GLU, dict(M=0)), (sg.sgemm_f32_glu, GLU, dict(F=0)),
    (sg.sgemm_f32_glu_bwd, BWD, dict(M=0, F=0)), (sg.sgemm_f32_glu_bwd, BWD, dict(K=0)),
    (sg.sgemm_f32_glu_bwd, BWD, dict(dX=0, dWg=0, dWu=0)),
    (sg.sgemm_f32_w4, W4, dict(M=0)), (sg.sgemm_f32_w4, W4, dict(F=0)),
    (sg.sgemm_f32_w4_glu, W4_GLU, dict(M=0)), (sg.sgemm_f32_w4_quantize, QUANT, dict(F=0)),
    (sg.sgemm_f32_w4_quantize, QUANT, dict(K=0)), (sg.sgemm_f32_w4_dequantize, DEQUANT, dict(F=0))],
    ids=lambda v: getattr(v, "__name__", None) or (None if isinstance(v, dict) and len(v) > 4 else str(v)))
def test_empty_outputs_touch_nothing(entry, good, empty):
    # null pointers everywhere: nothing would be read or written
    args = {k: 0 if v == P and k not in ("workspace",) else v for k, v in good.items()}
    assert entry(*dict(args, **empty).values(), stream=0) == 0


@pytest.mark.parametrize("entry,good", [(sg.sgemm_f32_glu, GLU), (sg.sgemm_f32_w4, W4)],
                         ids=lambda v: getattr(v, "__name__", "") or "args")
def test_sizes_beyond_the_index_range(entry, good):
    big = 1 << 40
    args = {k: big if k.startswith("ld") else v for k, v in good.items()}
    for name in ("M", "F", "K"):
        assert entry(*dict(args, **{name: (1 << 30) + 1}).values(), stream=0) == sg.ERR_TOO_LARGE


def test_workspace_size():
    for dtype, e in ((0, 4), (1, 2), (2, 2)):
        rc, n = sg.sgemm_f32_glu_bwd_ws_size(dtype, 100, 65, 30, 256)
        assert rc == 0 and n >= 2 * 100 * 128 * e
    assert sg.sgemm_f32_glu_bwd_ws_size(1, 0, 65, 30, 256) == (0, 0)
    assert sg.sgemm_f32_glu_bwd_ws_size(3, 1, 1, 1, 256)[0] == -17
    assert sg.sgemm_f32_glu_bwd_ws_size(0, -1, 1, 1, 256)[0] == -1
    assert sg.sgemm_f32_glu_bwd_ws_size(0, 1, 1, 1 << 31, 256)[0] == sg.ERR_TOO_LARGE
    from fp32_gemm_tuning_amd import ffn
    assert ffn._lib.sgemm_f32_glu_bwd_ws_size(0, 1, 1, 1, 256, None) == -12
    # 16-bit types: too little is refused before any launch
    need = sg.sgemm_f32_glu_bwd_ws_size(1, 4, 6, 8, 256)[1]
    assert sg.sgemm_f32_glu_bwd(*dict(BWD, dtype=1, workspace_bytes=need - 1).values(), stream=0) == sg.ERR_WORKSPACE
    assert sg.sgemm_f32_glu_bwd(*dict(BWD, dtype=1, workspace=0, workspace_bytes=0).values(),
                                stream=0) == sg.ERR_WORKSPACE


def test_helpers_refuse_what_they_cannot_pass():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        sg.glu(x, x, x)
    with pytest.raises(ValueError, match="2-D"):
        sg.glu(x[0], x, x)
    with pytest.raises(ValueError, match="group"):
        sg.ffn._groups(64, 33)
    from fp32_gemm_tuning_amd.ffn import _act, _dtype, _ld
    with pytest.raises(ValueError, match="activation"):
        _act("swish")
    with pytest.raises(TypeError, match="float32"):
        _dtype(x.double(), "X")
    with pytest.raises(TypeError, match="bfloat16"):
        _ld(x, x, torch.bfloat16, 4, 8, "Wg")
    with pytest.raises(ValueError, match="shape"):
        _ld(x, x, torch.float32, 8, 4, "Wg")
    with pytest.raises(ValueError, match="unit column stride"):
        _ld(x.t(), x, torch.float32, 8, 4, "Wg")
    with pytest.raises(ValueError, match="overlap"):
        _ld(x[:1].expand(4, 8), x, torch.float32, 4, 8, "Wg")
    assert _ld(x[:, :5], x, torch.float32, 4, 5, "Wg") == 8
    assert _ld(x[:1, :1], x, torch.float32, 1, 1, "Wg") == 1
    assert _ld(torch.zeros(4, 0), x, torch.float32, 4, 0, "Wg") == 1
