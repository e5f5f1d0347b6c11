"""The root-mean-square norm, its backward pass and matrices in 8 bits against
64-bit references (i8_ref.py), within bounds that count each rounding; whole
numbers of the 8-bit form are compared for equality. Operands sit in buffers
padded with NaN, which no result may show, and outputs in buffers whose
surroundings have to stay as they were."""
import pytest

torch = pytest.importorskip("torch")
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402
import i8_ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")


def _normal(shape, gen, dev, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * scale).to(dev, dtype)


def _gen(*seed):
    g = torch.Generator()
    g.manual_seed(hash(seed) & 0xFFFFFFFF)
    return g


def _say(*a):
    print("[gpu]", *a, flush=True)


def _out(rows, cols, dtype, dev, layout):
    return ref.laid_out(torch.full((rows, cols), float("nan"), dtype=dtype, device=dev), *layout)


def _out_q(rows, cols, dev, layout):
    return ref.laid_out(torch.full((rows, cols), 99, dtype=torch.int8, device=dev), *layout, fill=99)


def _out_vec(n, dev, dtype=torch.float32):
    """A vector inside a longer one of NaN."""
    flat = torch.full((n + 64,), float("nan"), dtype=dtype, device=dev)
    return flat[32:32 + n], flat


def _vec_kept(flat, n):
    return bool(torch.isnan(flat[:32]).all() and torch.isnan(flat[32 + n:]).all())


def _q_kept(flat, view):
    left = flat.clone()
    left.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(99)
    return bool((left == 99).all())


def _close(got, want, bound, what):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / bound).nan_to_num(nan=1e30).max()):.3g} of its bound, first at "
                           f"{bad.nonzero()[0].tolist()}")


# (M, K): single elements, rows of less than a 16-byte chunk, both sides of every
# power of two where another number of lanes or chunks may hold a row, rows too long
# for registers, and more rows than one workgroup's
SHAPES = [(1, 1), (3, 2), (5, 3), (4, 7), (2, 8), (5, 9), (70, 16), (9, 31), (5, 64), (4, 65), (7, 127), (9, 128),
          (6, 129), (33, 255), (8, 256), (5, 257), (5, 511), (5, 512), (17, 513), (3, 1000), (2, 1024), (3, 1025),
          (4, 2047), (2, 2048), (3, 2049), (3, 4096), (2, 4097), (1, 5000), (2, 8192), (3, 8200), (1, 16384),
          (2, 16385), (1, 32768), (2, 33001), (1, 65536), (2, 70001), (1100, 100), (600, 777), (300, 4100), (40, 16390)]
LAYOUTS = [(0, 0), (8, 8), (3, 1)]
EPS = 1e-5


def _inputs(shape, t, dev, seed, residual=True):
    """X, R and W: residual streams, some channels larger than the rest."""
    M, K = shape
    gen = _gen(seed, shape)
    big = torch.where(torch.rand(K, generator=gen) < 0.02, 20.0, 1.0).double()
    X, R = ((torch.randn((M, K), generator=gen, dtype=torch.float64) * big).to(dev, t) for _ in range(2))
    W = (1 + 0.3 * torch.randn(K, generator=gen, dtype=torch.float64)).to(dev, t)
    return X, R if residual else None, W


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rms_norm(dev, shape, dtype, layout):
    M, K = shape
    t = ref.DTYPES[dtype]
    _say("rms_norm", shape, dtype, layout)
    X, R, W = _inputs(shape, t, dev, 1)
    xs, rs = (ref.laid_out(v, *layout)[0] for v in (X, R))
    for r in (None, R):
        H = i8_ref.total(X, r)
        y, flat = _out(M, K, t, dev, layout)
        h, hflat = _out(M, K, t, dev, layout)
        rstd, rflat = _out_vec(M, dev)
        got = sg.rms_norm(xs, W, EPS, residual=None if r is None else rs, out=y, total=h, rstd=rstd)
        torch.cuda.synchronize()
        assert got is y and torch.equal(h, H)
        want = i8_ref.rstd(H, EPS)
        _close(rstd, want, want * (i8_ref.rstd_error(K) + 2.0 ** -24), "rstd")
        _close(y, i8_ref.norm(H, W, EPS), i8_ref.norm_bound(H, W, EPS, dtype), "Y")
        assert ref.around_untouched(flat, y) and ref.around_untouched(hflat, h) and _vec_kept(rflat, M)
        # without the extra outputs: the same bits
        assert torch.equal(sg.rms_norm(X, W, EPS, residual=r), y)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rms_norm_i8(dev, shape, dtype, layout):
    M, K = shape
    t = ref.DTYPES[dtype]
    _say("rms_norm_i8", shape, dtype, layout)
    X, R, W = _inputs(shape, t, dev, 2)
    xs, rs = (ref.laid_out(v, *layout)[0] for v in (X, R))
    for r in (None, R):
        H = i8_ref.total(X, r)
        q, qflat = _out_q(M, K, dev, layout)
        h, hflat = _out(M, K, t, dev, layout)
        s, sflat = _out_vec(M, dev)
        sg.rms_norm_i8(xs, W, EPS, residual=None if r is None else rs, out=sg.I8(q, s), total=h)
        torch.cuda.synchronize()
        v = H.double() * W.double()
        want, top = i8_ref.levels(v)
        sure = ~i8_ref.near_half(v, 2.0 ** -43) if dtype == "f32" else torch.ones_like(v, dtype=torch.bool)
        assert torch.equal(h, H) and torch.equal(q[sure], want[sure])
        scale = top / 127 * i8_ref.rstd(H, EPS)
        _close(s, scale, scale * (i8_ref.rstd_error(K) + 2.1 * 2.0 ** -24), "S")
        assert ref.around_untouched(hflat, h) and _q_kept(qflat, q) and _vec_kept(sflat, M)
        again = sg.rms_norm_i8(X, W, EPS, residual=r)
        assert torch.equal(again.q, q) and torch.equal(again.scales, s)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_i8_quantize(dev, shape, dtype, layout):
    M, K = shape
    t = ref.DTYPES[dtype]
    _say("i8_quantize", shape, dtype, layout)
    gen = _gen(3, shape)
    X = _normal((M, K), gen, dev, t)
    if M > 1:   # exact halves: quotients of a row whose largest number is 254
        X[1] = torch.randint(-254, 255, (K,), generator=gen).to(dev, t)
        X[1, K // 2] = 254
    q, qflat = _out_q(M, K, dev, layout)
    s, sflat = _out_vec(M, dev)
    sg.i8_quantize(ref.laid_out(X, *layout)[0], out=sg.I8(q, s))
    torch.cuda.synchronize()
    want, top = i8_ref.levels(X)
    assert torch.equal(q, want) and torch.equal(s, (top / 127).float())
    assert _q_kept(qflat, q) and _vec_kept(sflat, M)
    # and back, into a padded matrix of each type
    for name, o in ref.DTYPES.items():
        x, flat = _out(M, K, o, dev, layout)
        sg.i8_dequantize(sg.I8(q, s), out=x)
        assert torch.equal(x, (q.float() * s[:, None]).to(o)) and ref.around_untouched(flat, x)
        assert torch.equal(sg.i8_dequantize(sg.I8(q, s), o), x)


@pytest.mark.parametrize("K", [5, 100, 300, 3000, 20000, 70000])
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_rows_that_are_not_ordinary(dev, dtype, K):
    # Zeros, infinities and NaN, and values whose squares, products or quotients
    # leave FP32's range; each row by itself, between ordinary ones.
    t = ref.DTYPES[dtype]
    _say("rows not ordinary", dtype, K)
    gen = _gen(4, K)
    X = _normal((12, K), gen, dev, t)
    big, small = (30000.0, 2e-7) if dtype == "f16" else (2e38, 1e-38)
    X[1] = 0
    X[2, K // 2] = float("inf")
    X[3, -1] = float("nan")
    X[4, 0] = -float("inf")
    X[5] = (X[5].double().clamp(-1, 1) * big).to(t)
    X[6] = (X[6].double() * small).to(t)
    X[7] = 0
    X[7, K // 3] = torch.finfo(t).smallest_normal
    X[8] = big
    X[9] = (X[9].double() * (1e-30 if dtype != "f16" else 1e-5)).to(t)
    W = (1 + 0.3 * torch.randn(K, generator=gen, dtype=torch.float64)).to(dev, t)
    whole = torch.isfinite(X).all(1)
    # to 8 bits
    p = sg.i8_quantize(X)
    q, top = i8_ref.levels(X)
    assert torch.equal(p.q, q) and torch.equal(p.scales.isnan(), ~whole)
    _close(p.scales[whole], top[whole] / 127, (top[whole] / 127) * 2.0 ** -24 + 2.0 ** -149, "S")
    for eps in (1e-5, 0.0):
        rstd = torch.empty(12, device=dev)
        y = sg.rms_norm(X, W, eps, rstd=rstd)
        r = i8_ref.rstd(X, eps)
        assert (rstd[[2, 4]] == 0).all() and rstd[3].isnan() and (rstd[1].isinf() if eps == 0 else rstd[1] < 1e3)
        fine = whole & torch.isfinite(r) & (r < 3e38)
        _close(rstd[fine], r[fine], r[fine] * (i8_ref.rstd_error(K) + 2.0 ** -24) + 2.0 ** -149, "rstd")
        w = i8_ref.norm(X, W, eps)
        bound = i8_ref.norm_bound(X, W, eps, dtype)
        # (a subnormal rstd has lost bits; so has a product of such numbers)
        ok = fine & (r > 1.2e-38)
        _close(y[ok], w[ok], bound[ok], "Y")
        bad = torch.isinf(X)
        assert y[3].isnan().all() and (y[[2, 4]].isnan() == bad[[2, 4]]).all() and (y[[2, 4]][~bad[[2, 4]]] == 0).all()
        assert y[1].isnan().all() if eps == 0 else (y[1] == 0).all()
        p = sg.rms_norm_i8(X, W, eps)
        v = X.double() * W.double()
        q, top = i8_ref.levels(v)
        sure = ~i8_ref.near_half(v, 2.0 ** -43) if dtype == "f32" else torch.ones_like(v, dtype=torch.bool)
        sure |= ~whole[:, None] | (top == 0)[:, None]
        assert torch.equal(p.q[sure], q[sure]) and p.scales[~whole].isnan().all()
        s = top / 127 * r
        ok = fine & (r > 1.2e-38) & (s < 3e38)
        _close(p.scales[ok], s[ok], s[ok] * (i8_ref.rstd_error(K) + 3 * 2.0 ** -24) + 2.0 ** -149, "S")
        assert p.scales[1].isnan() if eps == 0 else p.scales[1] == 0


@pytest.mark.parametrize("K", [9, 200, 3000, 70000])
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_norm_weights_that_are_not_ordinary(dev, dtype, K):
    # An infinity or NaN in W stays in its column; in 8 bits it takes every row.
    t = ref.DTYPES[dtype]
    _say("weights not ordinary", dtype, K)
    X = _normal((3, K), _gen(5, K), dev, t)
    W = torch.ones(K, dtype=t, device=dev)
    plain = sg.rms_norm(X, W)
    W[K // 2], W[1] = float("nan"), float("inf")
    y = sg.rms_norm(X, W)
    at = torch.tensor([1, K // 2], device=dev)
    rest = torch.ones(K, dtype=torch.bool, device=dev)
    rest[at] = False
    assert torch.equal(y[:, rest], plain[:, rest]) and y[:, K // 2].isnan().all() and y[:, 1].isinf().all()
    p = sg.rms_norm_i8(X, W)
    assert p.scales.isnan().all() and (p.q == 0).all()


# ---------------------------------------------------------------------------
# Backward
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES + [(2500, 64), (1030, 2050), (20000, 24)], ids=lambda s: "x".join(map(str, s)))
def test_rms_norm_backward(dev, shape, dtype, layout):
    M, K = shape
    t = ref.DTYPES[dtype]
    _say("rms_norm_backward", shape, dtype, layout)
    H, D, W = _inputs(shape, t, dev, 6)
    dY = _normal((M, K), _gen(7, shape), dev, t)
    rstd = torch.empty(M, device=dev)
    sg.rms_norm(H, W, EPS, rstd=rstd)
    hs, ds, ys = (ref.laid_out(v, *layout)[0] for v in (H, D, dY))
    ws = torch.full((max(16, sg.rms_norm_backward_workspace(H)),), 0xFF, dtype=torch.uint8, device=dev)
    for d, strided in ((None, None), (D, ds)):
        dx, xflat = _out(M, K, t, dev, layout)
        dw, wflat = _out_vec(K, dev, t)
        got = sg.rms_norm_backward(ys, hs, W, rstd, dH=strided, dX=dx, dW=dw, workspace=ws)
        torch.cuda.synchronize()
        assert got[0] is dx and got[1] is dw
        want = i8_ref.norm_grads(dY, H, W, rstd, d)
        for name, a, b, c in zip(("dX", "dW"), got, want, i8_ref.norm_grads_bounds(dY, H, W, rstd, d, dtype)):
            _close(a, b, c, name)
        assert ref.around_untouched(xflat, dx) and _vec_kept(wflat, K)
        # either alone: the same bits
        only = sg.rms_norm_backward(dY, H, W, rstd, dH=d, dW=False)
        assert only[1] is None and torch.equal(only[0], dx)
        only = sg.rms_norm_backward(dY, H, W, rstd, dH=d, dX=False)
        assert only[0] is None and torch.equal(only[1], dw)


@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_backward_against_differences(dev, residual):
    # The slope of L = sum(dY Y) + sum(D H) along a direction, by central differences of
    # the 64-bit forward pass: with step h their error is h^2/6 times the third derivative
    # (below 1e3 here), 2^-53 |L| / h from rounding.
    M, K = 20, 130
    _say("rms_norm_backward differences", residual)
    gen = _gen(8)
    X, R, dY, D = (_normal((M, K), gen, dev, torch.float32) for _ in range(4))
    W = _normal((K,), gen, dev, torch.float32)
    r, h, y = torch.empty(M, device=dev), torch.empty_like(X), torch.empty_like(X)
    sg.rms_norm(X, W, EPS, residual=R if residual else None, out=y, total=h, rstd=r)
    dx, dw = sg.rms_norm_backward(dY, h, W, r, dH=D if residual else None)
    bounds = i8_ref.norm_grads_bounds(dY, h, W, r, D if residual else None, "f32")

    def loss(x, w):
        z = x + (R.double() if residual else 0)
        n = z / torch.sqrt((z * z).mean(1, keepdim=True) + EPS)
        return (dY.double() * n * w).sum() + ((D.double() * z).sum() if residual else 0)

    step = 1e-5
    at = [X.double(), W.double()]
    for i, (g, b) in enumerate(((dx, bounds[0]), (dw, bounds[1]))):
        d = torch.randn(g.shape, generator=gen, dtype=torch.float64).to(dev)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + step * d, at[i] - step * d
        slope = (loss(*up) - loss(*down)) / (2 * step)
        # (h and rstd are FP32 numbers: a rounding each, on what they multiply)
        extra = (g.double().abs() * d.abs()).sum() * 2.0 ** -21 + 1e-5
        assert abs((g.double() * d).sum() - slope) <= (b * d.abs()).sum() + extra, i


@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_gradients_of_rows_that_are_not_ordinary(dev, dtype):
    # An infinity or NaN in a row of dY or H stays in that row of dX; in dW, in its columns.
    t = ref.DTYPES[dtype]
    for K in (40, 3000, 70000):
        _say("gradients not ordinary", dtype, K)
        H, D, W = _inputs((6, K), t, dev, 9)
        dY = _normal((6, K), _gen(10, K), dev, t)
        rstd = torch.empty(6, device=dev)
        sg.rms_norm(H, W, EPS, rstd=rstd)
        plain = sg.rms_norm_backward(dY, H, W, rstd, dH=D)
        dY[2, 5], dY[4, 7] = float("inf"), float("nan")
        dx, dw = sg.rms_norm_backward(dY, H, W, rstd, dH=D)
        keep = torch.tensor([0, 1, 3, 5], device=dev)
        assert torch.equal(dx[keep], plain[0][keep]) and not torch.isfinite(dx[2]).any() and dx[4].isnan().all()
        rest = torch.ones(K, dtype=torch.bool, device=dev)
        rest[5] = rest[7] = False
        assert torch.equal(dw[rest], plain[1][rest]) and dw[5].isinf() and dw[7].isnan()


def test_empty_rows_and_no_rows(dev):
    _say("empty rows")
    for t in ref.DTYPES.values():
        e = lambda *s: torch.empty(*s, dtype=t, device=dev)   # noqa: E731
        r = torch.full((3,), float("nan"), device=dev)
        assert sg.rms_norm(e(3, 0), e(0), 0.25, rstd=r).shape == (3, 0) and (r == 2).all()
        p = sg.rms_norm_i8(e(3, 0), e(0), out=sg.I8(torch.empty(3, 0, dtype=torch.int8, device=dev),
                                                    torch.full((3,), float("nan"), device=dev)))
        assert (p.scales == 0).all()
        p = sg.i8_quantize(e(3, 0))
        assert (p.scales == 0).all() and sg.i8_dequantize(p, t).shape == (3, 0)
        assert sg.rms_norm(e(0, 5), e(5)).shape == (0, 5)
        dx, dw = sg.rms_norm_backward(e(0, 5), e(0, 5), e(5), torch.empty(0, device=dev),
                                      dW=torch.full((5,), float("nan"), dtype=t, device=dev))
        assert dx.shape == (0, 5) and (dw == 0).all()


# ---------------------------------------------------------------------------
# Memory
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("K", [100, 777, 4096, 8189, 16381, 20000, 70001])
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_outputs_in_place_of_inputs(dev, dtype, K):
    t = ref.DTYPES[dtype]
    _say("in place", dtype, K)
    X, R, W = _inputs((5, K), t, dev, 11)
    y, h = torch.empty_like(X), torch.empty_like(X)
    r = torch.empty(5, device=dev)
    sg.rms_norm(X, W, residual=R, out=y, total=h, rstd=r)
    q = sg.rms_norm_i8(X, W, residual=R)
    for where in ("X", "R"):
        x2, r2 = X.clone(), R.clone()
        mine = x2 if where == "X" else r2
        assert torch.equal(sg.rms_norm(x2, W, residual=r2, total=mine), y) and torch.equal(mine, h)
        x2, r2 = X.clone(), R.clone()
        mine, other = (x2, r2) if where == "X" else (r2, x2)
        sg.rms_norm(x2, W, residual=r2, total=other, out=mine)
        assert torch.equal(mine, y) and torch.equal(other, h)
        x2, r2 = X.clone(), R.clone()
        mine = x2 if where == "X" else r2
        sg.rms_norm(x2, W, residual=r2, out=mine)
        assert torch.equal(mine, y)
        x2, r2 = X.clone(), R.clone()
        mine = x2 if where == "X" else r2
        p = sg.rms_norm_i8(x2, W, residual=r2, total=mine)
        assert torch.equal(p.q, q.q) and torch.equal(p.scales, q.scales) and torch.equal(mine, h)
    x2 = X.clone()
    sg.rms_norm(x2, W, out=x2)
    assert torch.equal(x2, sg.rms_norm(X, W))
    dY, D = _normal((5, K), _gen(12, K), dev, t), R
    want = sg.rms_norm_backward(dY, h, W, r, dH=D)
    for where in ("dH", "dY"):
        d2, y2 = D.clone(), dY.clone()
        got = sg.rms_norm_backward(y2, h, W, r, dH=d2, dX=d2 if where == "dH" else y2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("K", [1027, 2051, 4099, 8195])
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_gradients_in_place_where_waves_share_elements(dev, dtype, K):
    # The last chunk of 16 bytes is moved back into the one that another wave of the workgroup holds and writes.
    t = ref.DTYPES[dtype]
    _say("gradients in place", dtype, K)
    H, D, W = _inputs((700, K), t, dev, 17)
    dY, r = _normal((700, K), _gen(18, K), dev, t), torch.rand(700, device=dev) + 0.5
    want = sg.rms_norm_backward(dY, H, W, r, dH=D)
    for where in ("dH", "dY"):
        d2, y2 = D.clone(), dY.clone()
        got = sg.rms_norm_backward(y2, H, W, r, dH=d2, dX=d2 if where == "dH" else y2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("K", [5, 100, 3000, 20000, 70001])
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_unusual_rows_in_place(dev, dtype, K):
    # The rows that are read again for each pass, written over their inputs: as when written elsewhere.
    t = ref.DTYPES[dtype]
    _say("unusual in place", dtype, K)
    X, R, W = _inputs((8, K), t, dev, 16)
    big, small = (30000.0, 2e-7) if dtype == "f16" else (2e38, 1e-38)
    for v in (X, R):
        v[1] = 0
        v[2, K // 2] = float("inf")
        v[3, 0] = float("nan")
        v[4] = (v[4].double().clamp(-0.4, 0.4) * big).to(t)
        v[5] = (v[5].double() * small).to(t)
    for eps in (1e-5, 0.0):
        y, h = torch.empty_like(X), torch.empty_like(X)
        sg.rms_norm(X, W, eps, residual=R, out=y, total=h)
        q = sg.rms_norm_i8(X, W, eps, residual=R)
        same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))   # noqa: E731 (NaN alike)
        for first in (True, False):
            x2, r2 = X.clone(), R.clone()
            mine, other = (x2, r2) if first else (r2, x2)
            sg.rms_norm(x2, W, eps, residual=r2, total=other, out=mine)
            assert same(mine, y) and same(other, h)
            x2, r2 = X.clone(), R.clone()
            mine = x2 if first else r2
            sg.rms_norm(x2, W, eps, residual=r2, out=mine)
            assert same(mine, y)
            x2, r2 = X.clone(), R.clone()
            mine = x2 if first else r2
            p = sg.rms_norm_i8(x2, W, eps, residual=r2, total=mine)
            assert same(p.q, q.q) and same(p.scales, q.scales) and same(mine, h)


@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_offsets_past_32_bits(dev, dtype):
    # Three rows of 2^31 elements and more apart, of which only their first ones are touched.
    t = ref.DTYPES[dtype]
    _say("far rows", dtype)
    K, ld = 300, (1 << 31) + 64
    X, R, W = _inputs((3, K), t, dev, 13)
    far = [torch.empty(2 * ld + K, dtype=t, device=dev).as_strided((3, K), (ld, 1)) for _ in range(2)]
    qf = torch.empty(2 * ld + K, dtype=torch.int8, device=dev).as_strided((3, K), (ld, 1))
    a, b = far
    r, s = torch.empty(3, device=dev), torch.empty(3, device=dev)
    a.copy_(X)
    sg.rms_norm(a, W, residual=R, total=a, out=b, rstd=r)
    h = i8_ref.total(X, R)
    y = sg.rms_norm(X, W, residual=R)
    assert torch.equal(a, h) and torch.equal(b, y)
    sg.rms_norm_i8(a, W, out=sg.I8(qf, s))
    near = sg.rms_norm_i8(h, W)
    assert torch.equal(qf, near.q) and torch.equal(s, near.scales)
    b.zero_()
    assert torch.equal(sg.i8_dequantize(sg.I8(qf, s), out=b), sg.i8_dequantize(near, t))
    sg.i8_quantize(a, out=sg.I8(qf, s))
    near = sg.i8_quantize(h)
    assert torch.equal(qf, near.q) and torch.equal(s, near.scales)
    dY = _normal((3, K), _gen(14), dev, t)
    want = sg.rms_norm_backward(dY, h, W, r, dH=R)
    b.copy_(dY)
    got = sg.rms_norm_backward(b, a, W, r, dH=R, dX=b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_many_rows(dev, dtype):
    t = ref.DTYPES[dtype]
    for M, K in ((1200000, 5), (300001, 33)):
        _say("many rows", dtype, M, K)
        X = torch.randint(-3, 4, (1, K), generator=_gen(15)).to(dev, t).expand(M, K).contiguous()
        X[M - 1] = torch.arange(K, device=dev).to(t)
        W = torch.ones(K, dtype=t, device=dev)
        y, p, s = sg.rms_norm(X, W), sg.rms_norm_i8(X, W), sg.i8_quantize(X)
        for got, few in ((y, sg.rms_norm(X[-2:], W)), (p.q, sg.rms_norm_i8(X[-2:], W).q),
                         (p.scales, sg.rms_norm_i8(X[-2:], W).scales), (s.q, sg.i8_quantize(X[-2:]).q),
                         (s.scales, sg.i8_quantize(X[-2:]).scales)):
            assert (got[:-1] == few[0]).all() and torch.equal(got[-1], few[1])
