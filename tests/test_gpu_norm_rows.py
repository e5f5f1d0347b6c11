"""The norm, its 8-bit form and matrices to 8 bits in more than 256 rows, where long
rows are held by fewer lanes in more chunks each: against 64-bit references (i8_ref.py),
written over their inputs, with rows that are not ordinary among others, and the
backward pass of such rows."""
import pytest

torch = pytest.importorskip("torch")
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402
import i8_ref  # noqa: E402
import test_gpu_norm as norm  # noqa: E402

pytestmark = pytest.mark.gpu

# Up to 512 chunks of 16 bytes a row is held the same way whatever the rows; 513 to 1024 chunks
# (16-bit K of 4097 to 8192, FP32 of 2049 to 4096) and 1025 to 2048 are not. Both ends of each
# range for both sizes of numbers, the last chunk moved back by each number of elements or not at all.
LONG = [2049, 2051, 4093, 4096, 4097, 4099, 5003, 8189, 8192, 8193, 8197, 16381, 16384]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")


@pytest.mark.parametrize("M", [256, 257])
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("K", LONG)
def test_against_the_definitions(dev, K, dtype, M):
    for layout in ((0, 0), (3, 1)):
        norm.test_rms_norm(dev, (M, K), dtype, layout)
        norm.test_rms_norm_i8(dev, (M, K), dtype, layout)
        norm.test_i8_quantize(dev, (M, K), dtype, layout)


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("K", [4099, 8195, 16381])
def test_backward_against_the_definition(dev, K, dtype):
    for layout in ((0, 0), (3, 1)):
        norm.test_rms_norm_backward(dev, (300, K), dtype, layout)


def _spoil(v, t):
    """Rows of zeros, infinities, NaN, and next to the ends of the range, wherever a workgroup's first and
    later rows are."""
    big, small = (30000.0, 2e-7) if t is torch.float16 else (2e38, 1e-38)
    for base in (0, 255, 280):
        v[base + 1] = 0
        v[base + 2, v.shape[1] // 2] = float("inf")
        v[base + 3, -1] = float("nan")
        v[base + 4] = (v[base + 4].double().clamp(-0.4, 0.4) * big).to(t)
        v[base + 5] = (v[base + 5].double() * small).to(t)


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))   # NaN alike


@pytest.mark.parametrize("unusual", [False, True])
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("K", LONG)
def test_outputs_in_place_of_inputs(dev, K, dtype, unusual):
    # Several waves hold a row, and a chunk moved back from its end is partly another wave's.
    t, M = ref.DTYPES[dtype], 300
    norm._say("in place, many rows", dtype, K, unusual)
    X, R, W = norm._inputs((M, K), t, dev, 21)
    if unusual:
        _spoil(X, t)
        _spoil(R, t)
    for eps in (1e-5, 0.0) if unusual else (1e-5,):
        y, h = torch.empty_like(X), torch.empty_like(X)
        sg.rms_norm(X, W, eps, residual=R, out=y, total=h)
        q = sg.rms_norm_i8(X, W, eps, residual=R)
        total = i8_ref.total(X, R)
        assert ((h == total) | (h.isnan() & total.isnan())).all()
        for first in (True, False):
            x2, r2 = X.clone(), R.clone()
            mine, other = (x2, r2) if first else (r2, x2)
            sg.rms_norm(x2, W, eps, residual=r2, total=other, out=mine)
            assert _same(mine, y) and _same(other, h)
            x2, r2 = X.clone(), R.clone()
            mine = x2 if first else r2
            assert _same(sg.rms_norm(x2, W, eps, residual=r2, total=mine), y) and _same(mine, h)
            x2, r2 = X.clone(), R.clone()
            mine = x2 if first else r2
            sg.rms_norm(x2, W, eps, residual=r2, out=mine)
            assert _same(mine, y)
            x2, r2 = X.clone(), R.clone()
            mine = x2 if first else r2
            p = sg.rms_norm_i8(x2, W, eps, residual=r2, total=mine)
            assert _same(p.q, q.q) and _same(p.scales, q.scales) and _same(mine, h)
        plain = sg.rms_norm(X, W, eps)
        x2 = X.clone()
        sg.rms_norm(x2, W, eps, out=x2)
        assert _same(x2, plain)
        x2 = X.clone()
        assert _same(sg.rms_norm(x2, W, eps, total=x2), plain) and _same(x2, X)


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("K", [2051, 4099, 8195, 16381])
def test_rows_that_are_not_ordinary(dev, K, dtype):
    # Those rows against the definitions; the rows beside them as without them.
    t, M = ref.DTYPES[dtype], 300
    norm._say("not ordinary, many rows", dtype, K)
    X, _, W = norm._inputs((M, K), t, dev, 22)
    before = sg.rms_norm(X, W), sg.rms_norm_i8(X, W), sg.i8_quantize(X)
    spoilt = torch.tensor([b + i for b in (0, 255, 280) for i in range(1, 6)], device=dev)
    kept = torch.ones(M, dtype=torch.bool, device=dev)
    kept[spoilt] = False
    _spoil(X, t)
    whole = torch.isfinite(X).all(1)
    y, p, s = sg.rms_norm(X, W), sg.rms_norm_i8(X, W), sg.i8_quantize(X)
    assert torch.equal(y[kept], before[0][kept])
    for now, old in ((p, before[1]), (s, before[2])):
        assert torch.equal(now.q[kept], old.q[kept]) and torch.equal(now.scales[kept], old.scales[kept])
    q, top = i8_ref.levels(X)
    assert torch.equal(s.q, q) and torch.equal(s.scales.isnan(), ~whole)
    v = X.double() * W.double()
    q, top = i8_ref.levels(v)
    sure = ~i8_ref.near_half(v, 2.0 ** -43) if dtype == "f32" else torch.ones_like(v, dtype=torch.bool)
    sure |= ~whole[:, None] | (top == 0)[:, None]
    assert torch.equal(p.q[sure], q[sure]) and p.scales[~whole].isnan().all()
    r = i8_ref.rstd(X, 1e-6)
    fine = whole & (r > 1.2e-38)      # (a subnormal rstd has lost bits)
    scale = (top / 127 * r)[fine]
    norm._close(p.scales[fine], scale, scale * (i8_ref.rstd_error(K) + 3 * 2.0 ** -24) + 2.0 ** -149, "S")
    norm._close(y[fine], i8_ref.norm(X, W, 1e-6)[fine], i8_ref.norm_bound(X, W, 1e-6, dtype)[fine], "Y")
    bad = torch.isinf(X)
    infinite = bad.any(1) & ~torch.isnan(X).any(1)
    assert (y[infinite].isnan() == bad[infinite]).all() and (y[infinite][~bad[infinite]] == 0).all()
    assert y[torch.isnan(X).any(1)].isnan().all() and (y[(X == 0).all(1)] == 0).all()
