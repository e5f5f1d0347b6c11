"""Every kernel of the products of matrices in 8 bits, each reached by name: scales
that are not powers of two and all four gates against 64-bit references (i8_ref.py), the
same bits as the kernels of few rows (which multiply scales in another
form), and scales next to the ends of FP32's range, zeros, infinities and NaN."""
import pytest

torch = pytest.importorskip("torch")
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402
import i8_ref  # noqa: E402

pytestmark = pytest.mark.gpu

# (kernel, (M, F, K)): sizes that no tile divides, K of whole 16-byte chunks for the kernels
# filled by buffer-to-LDS loads
DENSE = [("few 1", (1, 701, 1040)), ("few 2", (2, 701, 1043)), ("few 4", (3, 701, 1040)), ("few 8", (7, 701, 1043)),
         ("rows 32x32", (45, 333, 1040)), ("rows 32x32 through registers", (45, 333, 1043)),
         ("rows 32x64", (33, 4306, 144)), ("rows 32x64 through registers", (33, 4226, 181)),
         ("rows 64x64", (2758, 129, 192)), ("flat 64x64", (66, 5603, 145)), ("ring 64x128", (129, 5461, 208)),
         ("flat 64x128", (129, 5677, 163)), ("ring 128x128", (324, 5457, 144)), ("flat 128x128", (322, 5487, 178)),
         ("tile 128x128", (2312, 2583, 160)), ("flat 256x128", (710, 5502, 291)), ("tile 256x256", (2836, 4253, 144)),
         ("flat 256x256", (2183, 5474, 302)), ("tile 128x128 of short rows", (150, 301, 13))]
GATED = [("few 1", (1, 701, 1040)), ("few 2", (2, 701, 1043)), ("few 4", (3, 701, 1040)), ("few 8", (9, 133, 1043)),
         ("rows 32x64", (45, 333, 1040)), ("rows 32x64 through registers", (45, 333, 1043)),
         ("rows 64x64", (33, 4306, 144)), ("flat 64x64", (33, 4226, 181)), ("ring 64x128", (65, 4126, 192)),
         ("flat 64x128", (68, 4247, 159)), ("ring 128x128", (129, 5461, 208)), ("flat 128x128", (129, 5677, 163)),
         ("tile 128x128", (578, 4906, 192)), ("flat 256x128", (386, 4725, 306)), ("tile 256x256", (1284, 4430, 176)),
         ("flat 256x256", (1027, 5524, 261)), ("tile 128x128 of short rows", (150, 301, 13))]
# Sums of many slices, dense
SLICES = [("rows 32x32 through registers", (40, 200, 20001)), ("rows 32x32", (40, 200, 20000)),
          ("rows 64x64", (300, 2100, 9008)), ("flat 64x64", (300, 2100, 9001)), ("ring 64x128", (300, 4100, 2064)),
          ("ring 128x128", (520, 4100, 3088))]
FAR = "tile 64x64 of far rows"   # rows 2^23 bytes and more apart: test_rows_far_apart


def kernel(gated, x, w):
    """The kernel that a product of these matrices takes."""
    (M, K), F = x.shape, w.shape[0]
    row = lambda q: q.stride(0) if q.shape[0] > 1 else max(K, 1)   # noqa: E731
    return sg.sgemm_f32_i8_kernel(gated, M, F, K, x, row(x), w, row(w), w, row(w))


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")


def _say(*a):
    print("[gpu]", *a, flush=True)


def _gen(*seed):
    g = torch.Generator()
    g.manual_seed(hash(seed) & 0xFFFFFFFF)
    return g


def _matrix(rows, K, gen, dev, scale=1.0):
    q = torch.randint(-127, 128, (rows, K), generator=gen).to(dev, torch.int8)
    return sg.I8(q, ((torch.rand(rows, generator=gen) + 1e-3) * scale).to(dev))


def _operands(gated, name, shape, dev, seed):
    """x, wg and wu with random scales, sums times scales of the order of one."""
    M, F, K = shape
    gen = _gen(seed, shape)
    x, a, b = _matrix(M, K, gen, dev, 4.0 / 127 / 73 * K ** -0.5), _matrix(F, K, gen, dev), _matrix(F, K, gen, dev)
    assert kernel(gated, x.q, a.q) == name
    return x, a, b


def _close(got, want, bound, what):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / bound).nan_to_num(nan=1e30).max()):.3g} of its bound, first at "
                           f"{bad.nonzero()[0].tolist()}")


def _rows(x, n):
    return sg.I8(x.q[:n], x.scales[:n])


def _ids(v):
    return v.replace(" ", "_") if isinstance(v, str) else "x".join(map(str, v)) if isinstance(v, tuple) else None


@pytest.mark.parametrize("name,shape", DENSE, ids=_ids)
def test_random_scales(dev, name, shape):
    _say("kernel", name, shape)
    x, a, _ = _operands(0, name, shape, dev, 1)
    want = i8_ref.product(x, a)
    for dtype, t in ref.DTYPES.items():
        y = sg.i8_matmul(x, a, t)
        _close(y, want, i8_ref.product_bound(want, dtype), f"Y {dtype}")
        # a few rows of it by another kernel: the same bits
        for n in (1, 3, 20):
            if n < shape[0]:
                assert torch.equal(sg.i8_matmul(_rows(x, n), a, t), y[:n]), (dtype, n)
        few = sg.I8(a.q[:17], a.scales[:17])
        assert torch.equal(sg.i8_matmul(x, few, t), y[:, :17]), dtype


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("name,shape", GATED, ids=_ids)
def test_random_scales_and_gates(dev, name, shape, act):
    _say("kernel gated", name, shape, act)
    x, a, b = _operands(1, name, shape, dev, 2)
    want = i8_ref.glu(x, a, b, act)
    for dtype, t in ref.DTYPES.items():
        h = sg.i8_glu(x, a, b, act, t)
        _close(h, want, i8_ref.glu_bound(x, a, b, act, dtype), f"{act} {dtype}")
        for n in (1, 3, 20):
            if n < shape[0]:
                assert torch.equal(sg.i8_glu(_rows(x, n), a, b, act, t), h[:n]), (dtype, n)
        fa, fb = (sg.I8(w.q[:17], w.scales[:17]) for w in (a, b))
        assert torch.equal(sg.i8_glu(x, fa, fb, act, t), h[:, :17]), dtype


# Pairs of scales whose product is an ordinary number, and which FP32 holds while their product
# with a sum, taken one after the other, it may not.
PAIRS = [(2.0 ** -120, 2.0 ** 110), (2.0 ** 120, 2.0 ** -130), (2.0 ** -149, 2.0 ** 127), (2.0 ** 127, 2.0 ** -149)]


@pytest.mark.parametrize("gated,name,shape", [(0, *c) for c in DENSE] + [(1, *c) for c in GATED], ids=_ids)
def test_scales_that_are_not_ordinary(dev, gated, name, shape):
    _say("kernel scales", gated, name, shape)
    M, F, K = shape
    x, a, b = _operands(gated, name, shape, dev, 3)
    sums = x.q.double() @ a.q.double().T
    assert sums.abs().max() < 1 << 24             # FP32 numbers
    one = torch.ones_like(b.scales)

    def call(sx, sa, t=torch.float32):
        """Without a gate Y; with one relu(Y) U, U of ordinary scales."""
        if not gated:
            return sg.i8_matmul(sg.I8(x.q, sx), sg.I8(a.q, sa), t)
        return sg.i8_glu(sg.I8(x.q, sx), sg.I8(a.q, sa), sg.I8(b.q, one), "relu", t)

    if gated:
        us = x.q.double() @ b.q.double().T
    for i, j in PAIRS:
        got = call(torch.full((M,), i, device=dev), torch.full((F,), j, device=dev))
        want = (sums * i * j).float()
        if gated:   # U has X's scale too, and may leave FP32's range: so may the result
            want = want.clamp(min=0) * (us * i).float()
        assert torch.equal(got.nan_to_num(nan=7.0), want.nan_to_num(nan=7.0)), (i, j)
    # A few rows and columns whose scales are not ordinary, between others: the others keep their bits, which
    # in a tile's columns and rows beside them come from the other form of the product.
    sx, sa = x.scales.clone(), a.scales.clone()
    plain = {t: call(sx, sa, t) for t in ref.DTYPES.values()}
    cols = {c % F: v for c, v in ((3, 0.0), (5, float("inf")), (40, float("nan")), (F - 2, 2.0 ** 100),
                                  (70, 2.0 ** -140))}
    rows = {} if M < 3 else {1: float("nan"), M - 1: 2.0 ** -100}
    for c, v in cols.items():
        sa[c] = v
    for r, v in rows.items():
        sx[r] = v
    kept_c, kept_r = torch.ones(F, dtype=torch.bool, device=dev), torch.ones(M, dtype=torch.bool, device=dev)
    kept_c[list(cols)] = False
    kept_r[list(rows)] = False
    for dtype, t in ref.DTYPES.items():
        got = call(sx, sa, t)
        assert torch.equal(got[kept_r][:, kept_c], plain[t][kept_r][:, kept_c])
        some, at = got[kept_r], sums[kept_r]
        assert some[:, 40 % F].isnan().all() and (not rows or got[1].isnan().all())
        if gated:
            assert (some[:, 3] == 0).all()
            g = at[:, 5]      # inf * 0 is NaN, relu(-inf) is 0
            assert torch.equal(some[:, 5].isnan(), (g == 0) | ((g > 0) & (us[kept_r][:, 5] == 0)))
            assert (some[:, 5][g < 0] == 0).all()
        else:
            assert (some[:, 3] == 0).all() and torch.equal(some[:, 5].isnan(), at[:, 5] == 0)
            assert torch.equal(some[:, 5] == float("inf"), at[:, 5] > 0)
            # and the finite ones are the products of the definition
            fine = torch.isfinite(sa)
            want = i8_ref.product((x.q, sx), (a.q, sa))[kept_r][:, fine]
            over = want.abs() > torch.finfo(t).max
            bound = i8_ref.product_bound(want, dtype)
            _close(some[:, fine][~over], want[~over], bound[~over], f"finite scales {dtype}")
            assert torch.isinf(some[:, fine][over]).all()


@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_rows_far_apart(dev, dtype):
    # Weight rows of 2^23 bytes and more: the tile with 64-bit addresses.
    _say("kernel far", dtype)
    t, (M, F, K), ld = ref.DTYPES[dtype], (70, 65, 300), (1 << 23) + 48
    gen = _gen(4)
    x, a, b = (_matrix(r, K, gen, dev, s) for r, s in ((M, 4.0 / 127 / 73 * K ** -0.5), (F, 1.0), (F, 1.0)))
    far = [sg.I8(torch.full(((F - 1) * ld + K,), 113, dtype=torch.int8, device=dev).as_strided((F, K), (ld, 1)), w.scales)
           for w in (a, b)]
    for f, w in zip(far, (a, b)):
        f.q.copy_(w.q)
    for g in (0, 1):
        assert kernel(g, x.q, far[0].q) == FAR
    want = i8_ref.product(x, a)
    y = sg.i8_matmul(x, far[0], t)
    _close(y, want, i8_ref.product_bound(want, dtype), "Y")
    assert torch.equal(y, sg.i8_matmul(x, a, t))
    for act in ref.ACTS:
        h = sg.i8_glu(x, *far, act, t)
        _close(h, i8_ref.glu(x, a, b, act), i8_ref.glu_bound(x, a, b, act, dtype), act)
        assert torch.equal(h, sg.i8_glu(x, a, b, act, t))
    assert all(bool((f.q.as_strided((F - 1, 64), (ld, 1), K) == 113).all()) for f in far)


@pytest.mark.parametrize("name,shape", SLICES, ids=_ids)
def test_many_slices_that_differ(dev, name, shape):
    # Each slice of 128 k has numbers of its own size, so that one read twice, or late, shows.
    _say("kernel slices", name, shape)
    M, F, K = shape
    gen = _gen(5)
    size = 1 + (torch.arange(K) // 128 * 37) % 61
    x, w = ((torch.randint(-2, 3, (r, K), generator=gen) * size).to(dev, torch.int8) for r in (M, F))
    assert kernel(0, x, w) == name
    s = [torch.ones(r, device=dev) for r in (M, F)]
    want = (x.double() @ w.double().T).float()
    for _ in range(3):
        assert torch.equal(sg.i8_matmul(sg.I8(x, s[0]), sg.I8(w, s[1])), want)
