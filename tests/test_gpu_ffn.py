"""The gated feed-forward block, its backward pass and products with 4-bit
weights against 64-bit references (ffn_ref.py).

Whole-number inputs are checked bit for bit: every sum is then exact in FP32
in any order, so a result is the exact value rounded once to the type.
Random inputs are checked within bounds that count each rounding. Operands
sit in buffers padded with NaN, which no result may show, and outputs in
buffers whose surroundings have to stay as they were."""
import pytest

torch = pytest.importorskip("torch")
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")


def _ints(shape, gen, lo, hi, dev, dtype):
    return torch.randint(lo, hi + 1, shape, generator=gen).to(dev, dtype)


def _normal(shape, gen, dev, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * scale).to(dev, dtype)


def _gen(*seed):
    g = torch.Generator()
    g.manual_seed(hash(seed) & 0xFFFFFFFF)
    return g


def _say(*a):
    print("[gpu]", *a, flush=True)


def _out(rows, cols, dtype, dev, pad=0, offset=0):
    return ref.laid_out(torch.full((rows, cols), float("nan"), dtype=dtype, device=dev), pad, offset)


# (M, F, K): single elements, tails in each direction, whole tiles and more
# than one tile of every kernel
SHAPES = [(1, 1, 1), (1, 7, 1000), (2, 300, 8), (3, 65, 31), (5, 64, 64), (16, 96, 256), (17, 33, 65),
          (32, 130, 520), (33, 64, 72), (64, 128, 128), (70, 31, 513), (128, 64, 192), (129, 257, 191),
          (300, 200, 77), (257, 512, 64), (2, 9, 2), (4, 17, 3), (6, 40, 3), (12, 3800, 90), (9, 8200, 40),
          (2, 33, 2100)]
# (pad, offset) of every operand's rows, in elements
LAYOUTS = [(0, 0), (8, 8), (3, 1)]


def _close(got, want, bound, what):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / bound).nan_to_num(nan=1e30).max()):.3g} of its bound, first at "
                           f"{bad.nonzero()[0].tolist()}")


# ---------------------------------------------------------------------------
# The gated block
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_glu_whole_numbers(dev, shape, dtype, layout):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    _say("glu ints", shape, dtype, layout)
    gen = _gen(1, shape)
    X, Wg, Wu = (_ints(s, gen, -2, 2, dev, t) for s in ((M, K), (F, K), (F, K)))
    xs, gs, us = (ref.laid_out(x, *layout)[0] for x in (X, Wg, Wu))
    H, flat = _out(M, F, t, dev, *layout)
    P, pflat = _out(M, 2 * F, torch.float32, dev, *layout)
    sg.glu(xs, gs, us, "relu", out=H, preact=P)
    torch.cuda.synchronize()
    g, u = X.double() @ Wg.double().T, X.double() @ Wu.double().T
    assert torch.equal(P.double(), torch.cat((g, u), 1))
    assert torch.equal(H, (g.clamp(min=0) * u).to(t))
    assert ref.around_untouched(flat, H) and ref.around_untouched(pflat, P)
    H2 = sg.glu(xs, gs, us, "relu")            # without the pre-activations: the same bits
    assert torch.equal(H2, H)


# Enough tiles for the largest block tile in each product (H: M x 2F, dX:
# M x K, dW: F x K) with ragged edges in whole 16-byte chunks, products
# split over their slices (few tiles, long sums), and odd ones of both kinds.
LARGE = [(3000, 4136, 144), (2904, 72, 4200), (72, 2600, 2728), (520, 264, 200), (100, 3001, 130),
         (2500, 65, 67), (1201, 1203, 1205), (2050, 2048, 8)]


@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large_whole_numbers(dev, shape, dtype):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    _say("large ints", shape, dtype)
    gen = _gen(14, shape)
    X, Wg, Wu, dH = (_ints(s, gen, -1, 1, dev, t) for s in ((M, K), (F, K), (F, K), (M, F)))
    H, flat = _out(M, F, t, dev, 8, 8)
    sg.glu(X, Wg, Wu, "relu", out=H)
    x, wg, wu, dh = (v.double() for v in (X, Wg, Wu, dH))
    g, u = x @ wg.T, x @ wu.T
    assert torch.equal(H, (g.clamp(min=0) * u).to(t)) and ref.around_untouched(flat, H)
    got = _backward(dH, X, Wg, Wu, "relu", (0, 0), dev)
    dg, du = (dh * u * (g > 0)).to(t).double(), (dh * g.clamp(min=0)).to(t).double()
    for name, a, b in zip(("dX", "dWg", "dWu"), got, (dg @ wg + du @ wu, dg.T @ x, du.T @ x)):
        assert torch.equal(a, b.to(t)), name


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", [(1, 64, 256), (9, 130, 77), (200, 150, 300)], ids=str)
def test_glu_random(dev, shape, dtype, act):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    _say("glu random", shape, dtype, act)
    gen = _gen(2, shape)
    X = _normal((M, K), gen, dev, t, 2.0)
    Wg, Wu = (_normal((F, K), gen, dev, t, K ** -0.5) for _ in range(2))
    H = sg.glu(X, Wg, Wu, act)
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    _close(H, ref.glu(x, wg, wu, act), ref.glu_bound(x, wg, wu, act, dtype), act)


@pytest.mark.parametrize("act", ref.ACTS)
def test_glu_far_arguments(dev, act):
    # G from -200 to 200, and infinite or NaN inputs: U is 1, so H is act(G).
    _say("glu far", act)
    g = torch.tensor([-200.0, -90.0, -30.0, -10.0, -1.0, -0.0, 0.0, 1e-30, 1.0, 10.0, 90.0, 200.0], device=dev)
    X = torch.stack((g, torch.ones_like(g)), 1).contiguous()
    Wg = torch.tensor([[1.0, 0.0]], device=dev)
    Wu = torch.tensor([[0.0, 1.0]], device=dev)
    H = sg.glu(X, Wg, Wu, act)
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    _close(H, ref.glu(x, wg, wu, act), ref.glu_bound(x, wg, wu, act, "f32"), act)
    X = torch.tensor([[float("inf"), 1.0], [float("nan"), 1.0], [2.0, 1.0]], device=dev)
    H = sg.glu(X, torch.tensor([[1.0, 1.0]], device=dev), torch.tensor([[1.0, 1.0]], device=dev), act)
    assert H[0, 0] == float("inf") and torch.isnan(H[1, 0]) and torch.isfinite(H[2, 0])   # rows stay apart


# ---------------------------------------------------------------------------
# Its backward pass
# ---------------------------------------------------------------------------
def _backward(dH, X, Wg, Wu, act, layout, dev):
    """(dX, dWg, dWu) through padded operands, checking the surroundings."""
    t = X.dtype
    M, K = X.shape
    F = Wg.shape[0]
    xs, gs, us, hs = (ref.laid_out(v, *layout)[0] for v in (X, Wg, Wu, dH))
    P, _ = _out(M, 2 * F, torch.float32, dev, *layout)
    sg.glu(xs, gs, us, act, preact=P)
    outs = [_out(r, K, t, dev, *layout) for r in (M, F, F)]
    ws = torch.full((max(16, sg.glu_backward_workspace(xs, F)),), 0xFF, dtype=torch.uint8, device=dev)
    got = sg.glu_backward(hs, xs, gs, us, P, act, *(o[0] for o in outs), workspace=ws)
    torch.cuda.synchronize()
    for (o, flat), g in zip(outs, got):
        assert g is o and ref.around_untouched(flat, o)
    return got


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_glu_backward_whole_numbers(dev, shape, dtype, layout):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    _say("glu_backward ints", shape, dtype, layout)
    gen = _gen(3, shape)
    X, Wg, Wu, dH = (_ints(s, gen, -1, 1, dev, t) for s in ((M, K), (F, K), (F, K), (M, F)))
    got = _backward(dH, X, Wg, Wu, "relu", layout, dev)
    x, wg, wu, dh = (v.double() for v in (X, Wg, Wu, dH))
    g, u = x @ wg.T, x @ wu.T
    dg, du = (dh * u * (g > 0)).to(t).double(), (dh * g.clamp(min=0)).to(t).double()   # rounded once
    for name, a, b in zip(("dX", "dWg", "dWu"), got, (dg @ wg + du @ wu, dg.T @ x, du.T @ x)):
        assert torch.equal(a, b.to(t)), name


@pytest.mark.parametrize("act", ref.ACTS[:3])
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", [(1, 64, 256), (1, 3620, 87), (9, 130, 77), (128, 128, 40), (129, 128, 40),
                                   (200, 150, 300)], ids=str)
def test_glu_backward_random(dev, shape, dtype, act):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    _say("glu_backward random", shape, dtype, act)
    gen = _gen(4, shape)
    X, dH = _normal((M, K), gen, dev, t, 2.0), _normal((M, F), gen, dev, t)
    Wg, Wu = (_normal((F, K), gen, dev, t, K ** -0.5) for _ in range(2))
    got = _backward(dH, X, Wg, Wu, act, (0, 0), dev)
    args = [v.double() for v in (dH, X, Wg, Wu)]
    for name, a, b, c in zip(("dX", "dWg", "dWu"), got, ref.glu_grads(*args, act),
                             ref.glu_grads_bounds(*args, act, dtype)):
        _close(a, b, c, name)


@pytest.mark.parametrize("act", ref.ACTS[:3])
def test_glu_backward_against_differences(dev, act):
    # The slope of L = sum(dH * H) along a direction, by central differences
    # of the 64-bit forward pass: with step h their error is h^2/6 times the
    # third derivative (below 1e3 here), 2^-53 |L| / h from rounding.
    M, F, K = 20, 33, 40
    _say("glu_backward differences", act)
    gen = _gen(5)
    X, dH = _normal((M, K), gen, dev, torch.float32), _normal((M, F), gen, dev, torch.float32)
    Wg, Wu = (_normal((F, K), gen, dev, torch.float32, K ** -0.5) for _ in range(2))
    grads = _backward(dH, X, Wg, Wu, act, (0, 0), dev)
    at = [v.double() for v in (X, Wg, Wu)]
    bounds = ref.glu_grads_bounds(dH.double(), *at, act, "f32")
    h = 1e-5
    for i, (g, b) in enumerate(zip(grads, bounds)):
        d = torch.randn(g.shape, generator=gen, dtype=torch.float64).to(dev)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * d, at[i] - h * d
        slope = (dH.double() * (ref.glu(*up, act) - ref.glu(*down, act))).sum() / (2 * h)
        assert abs((g.double() * d).sum() - slope) <= (b * d.abs()).sum() + 1e-6, i


@pytest.mark.parametrize("shape", [(40, 70, 90), (1500, 200, 300), (300, 1500, 1200)], ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_glu_backward_parts(dev, dtype, shape):
    # Any of the three alone gives the same bits as all of them.
    t = ref.DTYPES[dtype]
    M, F, K = shape
    _say("glu_backward parts", dtype, shape)
    gen = _gen(6, shape)
    X, dH = _normal((M, K), gen, dev, t), _normal((M, F), gen, dev, t)
    Wg, Wu = (_normal((F, K), gen, dev, t, 0.1) for _ in range(2))
    P = torch.empty(M, 2 * F, device=dev)
    sg.glu(X, Wg, Wu, preact=P)
    every = sg.glu_backward(dH, X, Wg, Wu, P)
    for keep in range(3):
        only = [None if i == keep else False for i in range(3)]
        part = sg.glu_backward(dH, X, Wg, Wu, P, dX=only[0], dWg=only[1], dWu=only[2])
        assert [p is None for p in part] == [i != keep for i in range(3)]
        assert torch.equal(part[keep], every[keep])


def test_empty_sums(dev):
    _say("empty sums")
    for t in ref.DTYPES.values():
        e = lambda r, c: torch.empty(r, c, dtype=t, device=dev)   # noqa: E731
        nan = lambda r, c: torch.full((r, c), float("nan"), dtype=t, device=dev)   # noqa: E731
        P = torch.full((3, 10), float("nan"), device=dev)
        H = sg.glu(e(3, 0), e(5, 0), e(5, 0), out=nan(3, 5), preact=P)
        assert (H == 0).all() and (P == 0).all()
        assert sg.glu(e(0, 4), nan(5, 4), nan(5, 4)).shape == (0, 5)
        dx, dg, du = sg.glu_backward(e(0, 5), e(0, 4), nan(5, 4), nan(5, 4), torch.empty(0, 10, device=dev),
                                     dWg=nan(5, 4), dWu=nan(5, 4))
        assert dx.shape == (0, 4) and (dg == 0).all() and (du == 0).all()
        dx, dg, du = sg.glu_backward(e(3, 0), nan(3, 4), e(0, 4), e(0, 4), torch.empty(3, 0, device=dev),
                                     dX=nan(3, 4))
        assert (dx == 0).all() and dg.shape == (0, 4) and du.shape == (0, 4)
        w = sg.w4_quantize(e(5, 0), 32)
        assert w.q.shape == (5, 0)
        assert (sg.w4_matmul(e(3, 0), w, out=nan(3, 5)) == 0).all()
        assert (sg.w4_glu(e(3, 0), w, w, out=nan(3, 5)) == 0).all()


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
# (F, K, group)
PACKS = [(1, 1, 32), (3, 31, 32), (5, 33, 32), (7, 777, 64), (64, 256, 128), (33, 100, 1000), (16, 130, 96),
         (20, 519, 256), (6, 1300, 512), (5, 1100, 1024)]


@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("pack", PACKS, ids=str)
def test_w4_quantize(dev, pack, dtype, zeros):
    F, K, group = pack
    t = ref.DTYPES[dtype]
    _say("w4_quantize", pack, dtype, zeros)
    gen = _gen(7, pack)
    W = _normal((F, K), gen, dev, t)
    W[0] = 0                                   # a row of zeros: scale 0
    W[-1] = W[-1].abs()                        # one sign only
    if F > 4:
        W[4] = (W[4].double() * (2e-40 if dtype == "f32" else 1e-6)).to(t)    # scales next to 0, or 0
    if F > 3:
        W[1] = _ints((K,), gen, -7, 7, dev, t) * 0.5      # quotients on whole and half steps
        W[2, K // 2] = float("inf")
        W[3, -1] = float("nan")
    ws = ref.laid_out(W, 3, 1)[0]
    w = sg.w4_quantize(ws, group, zeros=zeros)
    q, s, z = ref.quantise(W.cpu(), group, zeros, t)
    assert torch.equal(w.scales.cpu().nan_to_num(nan=-1), s.nan_to_num(nan=-1))
    assert (w.zeros is None) == (not zeros) and (not zeros or torch.equal(w.zeros.cpu(), z))
    n, m = (torch.stack((v & 15, v >> 4), -1).reshape(F, -1) for v in (w.q.cpu(), q))
    fine = torch.isfinite(s).repeat_interleave(group, 1)[:, :K]
    assert torch.equal(n[:, :K][fine], m[:, :K][fine]) and (K % 2 == 0 or (n[:, K] == 0).all())
    # and back, into a padded matrix
    out, flat = _out(F, K, t, dev, 3, 1)
    sg.w4_dequantize(w, out=out)
    want = ref.w4_values(w.q, w.scales, w.zeros, K, group).to(t)
    assert torch.equal(out.nan_to_num(nan=-1), want.nan_to_num(nan=-1)) and torch.isnan(out).any() == (F > 3)
    if F <= 3:
        assert ref.around_untouched(flat, out)


def _packed(F, K, group, zeros, gen, dev, t, exact, pad):
    """Random 4-bit weights in padded matrices; with `exact`, power-of-two
    scales and whole zero points."""
    G, B = -(-K // group), (K + 1) // 2
    q = torch.randint(0, 256, (F, B), generator=gen).to(dev, torch.uint8)
    qs = ref.laid_out(q, pad, pad, fill=255)[0]
    if exact:
        s = (2.0 ** torch.randint(-1, 2, (F, G), generator=gen)).to(dev, t)
        z = _ints((F, G), gen, 0, 15, dev, t)
    else:
        s = (torch.rand((F, G), generator=gen) * K ** -0.5 / 8 + 1e-3).to(dev, t)
        z = (torch.rand((F, G), generator=gen) * 15).to(dev, t)
    ss, zs = ref.laid_out(s, pad, pad)[0], ref.laid_out(z, pad, pad)[0]
    return sg.W4(qs, ss, zs if zeros else None, K, group)


W4_SHAPES = [(1, 1, 1, 32), (1, 48, 256, 32), (1, 17, 1000, 128), (2, 100, 77, 64), (3, 33, 520, 32),
             (4, 64, 4096, 256), (5, 65, 31, 32), (6, 40, 384, 96), (16, 96, 640, 64), (17, 130, 129, 32),
             (33, 50, 300, 1000), (64, 70, 512, 128), (65, 16, 96, 32), (130, 130, 130, 32), (200, 33, 64, 64),
             (48, 20, 1100, 64), (90, 36, 700, 128), (3, 20, 8200, 128), (16, 33, 9000, 32),
             (250, 4090, 1100, 64), (130, 8200, 321, 32), (32, 16390, 200, 128), (256, 4100, 1536, 256), (150, 4090, 321, 32),
             (60, 8190, 200, 64), (60, 4090, 130, 96)]


@pytest.mark.parametrize("pad", [0, 16, 3])
@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", W4_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_w4_whole_numbers(dev, shape, dtype, zeros, pad):
    M, F, K, group = shape
    t = ref.DTYPES[dtype]
    _say("w4 ints", shape, dtype, zeros, pad)
    gen = _gen(8, shape, zeros)
    X = _ints((M, K), gen, -3, 3, dev, t)
    xs = ref.laid_out(X, pad, pad)[0]
    wg, wu = (_packed(F, K, group, zeros, gen, dev, t, True, pad) for _ in range(2))
    g, u = (X.double() @ ref.w4_values(*w).T for w in (wg, wu))
    Y, flat = _out(M, F, t, dev, pad, pad)
    sg.w4_matmul(xs, wg, out=Y)
    assert torch.equal(Y, g.to(t)) and ref.around_untouched(flat, Y)
    H, flat = _out(M, F, t, dev, pad, pad)
    sg.w4_glu(xs, wg, wu, "relu", out=H)
    # the product of two exact sums, rounded to FP32 and then to the type
    want = (g.clamp(min=0) * u).float().to(t)
    assert torch.equal(H, want) and ref.around_untouched(flat, H)


@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", [(1, 40, 1024, 128), (7, 33, 777, 32), (40, 64, 300, 64), (100, 20, 2048, 256)],
                         ids=str)
def test_w4_random(dev, shape, dtype, zeros):
    M, F, K, group = shape
    t = ref.DTYPES[dtype]
    _say("w4 random", shape, dtype, zeros)
    gen = _gen(9, shape)
    X = _normal((M, K), gen, dev, t)
    X[0] = X[0].abs()                          # one sign: the sums of x are large
    w = [_packed(F, K, group, zeros, gen, dev, t, False, 0) for _ in range(2)]
    x = X.double()
    (g, u), (b0, b1) = zip(*((x @ ref.w4_values(*v).T, ref.w4_bound(x, *v, dtype)) for v in w))
    _close(sg.w4_matmul(X, w[0]), g, b0[1], "w4")
    for act in ref.ACTS:
        a = ref.act(g, act)[0]
        e = 1.13 * b0[0] * (u.abs() + b1[0]) + a.abs() * b1[0]
        e = e + (a * u).abs() * (ref.act_eval_error(g, act) + 2.0 ** -23)
        e = e + ref.HALF_STEP[dtype] * ((a * u).abs() + e) + ref.TINY[dtype]
        _close(sg.w4_glu(X, *w, act), a * u, e, act)


@pytest.mark.parametrize("M", [9, 200])
@pytest.mark.parametrize("zeros", [False, True], ids=["symmetric", "zeros"])
def test_w4_keeps_single_precision(dev, zeros, M):
    """One group, |x| in [1/2, 2): the sums of 8-bit leading parts are exact
    (93 * 31 * 2 < 2^13, in steps of 2^-8), so three roundings of results remain
    (the zero point's, the rest's and the scale's), at most 2^-24 each in the norm, and
    those of the rest's sums, 2^-7 of the products: 4 * 2^-24 in all."""
    gen = _gen(21, M, zeros)
    _say("w4 fp32", M, zeros)
    X = torch.rand(M, 93, generator=gen) * 1.5 + 0.5
    X = (X * torch.where(torch.rand(M, 93, generator=gen) < 0.5, -1.0, 1.0)).to(dev)
    w = sg.w4_quantize(torch.randn(97, 93, generator=gen).to(dev), 256, zeros)
    want = X.double() @ ref.w4_values(*w).T
    got = sg.w4_matmul(X, w).double()
    assert float((got - want).norm() / want.norm()) <= 4 * 2.0 ** -24


def test_w4_rows_stay_apart(dev):
    # NaN and infinities in one row of X, and a NaN scale in one row of W,
    # show in that row and column only.
    _say("w4 rows apart")
    for t in ref.DTYPES.values():
        gen = _gen(10)
        for M in (1, 3, 16, 40):
            X = _ints((M, 256), gen, -3, 3, dev, t)
            w = _packed(48, 256, 64, True, gen, dev, t, True, 0)
            Y = sg.w4_matmul(X, w)
            X[M // 2, 100] = float("nan")
            w.scales[7, 3] = float("nan")
            Y2 = sg.w4_matmul(X, w)
            assert torch.isnan(Y2[M // 2]).all() and torch.isnan(Y2[:, 7]).all()
            rows = [m for m in range(M) if m != M // 2]
            cols = [c for c in range(48) if c != 7]
            assert torch.equal(Y2[rows][:, cols], Y[rows][:, cols])


# ---------------------------------------------------------------------------
# Together, and as a program calls them
# ---------------------------------------------------------------------------
def test_train_pack_and_serve(dev):
    # One layer in single precision: a step of gradient descent, the weights
    # packed, tokens served through the packed block and a packed projection
    # down, against 64 bits over the values the packed weights stand for.
    _say("train, pack, serve")
    M, F, K = 48, 160, 96
    gen = _gen(11)
    X, dH = _normal((M, K), gen, dev, torch.float32), _normal((M, F), gen, dev, torch.float32)
    Wg, Wu = (_normal((F, K), gen, dev, torch.float32, K ** -0.5) for _ in range(2))
    Wd = _normal((K, F), gen, dev, torch.float32, F ** -0.5)
    P = torch.empty(M, 2 * F, device=dev)
    H = sg.glu(X, Wg, Wu, preact=P)
    Y = torch.empty(M, K, device=dev)
    sg.gemm(H, Wd.t(), Y)
    _, dWg, dWu = sg.glu_backward(dH, X, Wg, Wu, P, dX=False)
    Wg, Wu = Wg - 0.01 * dWg, Wu - 0.01 * dWu
    wg, wu, wd = (sg.w4_quantize(w, 32) for w in (Wg, Wu, Wd))
    vg, vu, vd = (ref.w4_values(*w) for w in (wg, wu, wd))
    for tokens in (1, 5, M):
        x = X[:tokens].contiguous()
        h = sg.w4_glu(x, wg, wu)
        _close(h, ref.glu(x.double(), vg, vu, "silu"),
               ref.w4_bound(x.double(), *wg, "f32")[1] * 100 + 1e-4, "w4_glu")
        y = sg.w4_matmul(h, wd)
        _close(y, h.double() @ vd.T, ref.w4_bound(h.double(), *wd, "f32")[1], "w4")
        # a prompt through the expanded weights and the dense product gives the same
        z = torch.empty(tokens, K, device=dev)
        sg.gemm(h, sg.w4_dequantize(wd).t(), z)
        _close(z, h.double() @ vd.T, ref.w4_bound(h.double(), *wd, "f32")[1], "gemm")


@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_graph_replays_match_eager(dev, dtype):
    t = ref.DTYPES[dtype]
    _say("graph", dtype)
    M, F, K = 70, 200, 136
    gen = _gen(12)
    X, dH = _normal((M, K), gen, dev, t), _normal((M, F), gen, dev, t)
    Wg, Wu = (_normal((F, K), gen, dev, t, 0.1) for _ in range(2))
    outs = [torch.empty(s, dtype=t, device=dev) for s in ((M, F), (M, K), (F, K), (F, K), (M, F), (M, F))]
    P = torch.empty(M, 2 * F, device=dev)
    ws = torch.empty(sg.glu_backward_workspace(X, F), dtype=torch.uint8, device=dev)
    w = sg.w4_quantize(Wg, 32, zeros=True)

    def step():
        sg.glu(X, Wg, Wu, out=outs[0], preact=P)
        sg.glu_backward(dH, X, Wg, Wu, P, dX=outs[1], dWg=outs[2], dWu=outs[3], workspace=ws)
        sg.w4_matmul(X, w, out=outs[4])
        sg.w4_glu(X, w, w, out=outs[5])

    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    eager = [o.clone() for o in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for r in range(4):
        for o in outs:
            o.fill_(float("nan"))
        P.fill_(float("nan"))
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager)), r
        sg.glu(X[:3], Wg, Wu)              # eager work between the replays
        torch.cuda.synchronize()
    del g


def test_two_streams(dev):
    # Two calls of different sizes at once, each with a workspace of its own.
    _say("two streams")
    gen = _gen(13)
    t = torch.bfloat16
    jobs = []
    for M, F, K in ((300, 500, 260), (190, 260, 700)):
        X, dH = _normal((M, K), gen, dev, t), _normal((M, F), gen, dev, t)
        Wg, Wu = (_normal((F, K), gen, dev, t, 0.1) for _ in range(2))
        P = torch.empty(M, 2 * F, device=dev)
        sg.glu(X, Wg, Wu, preact=P)
        jobs.append((dH, X, Wg, Wu, P))
    alone = [sg.glu_backward(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in jobs]
    outs = [[torch.empty_like(g) for g in a] for a in alone]
    spaces = [torch.empty(sg.glu_backward_workspace(j[1], j[2].shape[0]), dtype=torch.uint8, device=dev)
              for j in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        for j, o, w, s in zip(jobs, outs, spaces, streams):
            sg.glu_backward(*j, dX=o[0], dWg=o[1], dWu=o[2], workspace=w, stream=s)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(x, y) for x, y in zip(a, o))


def test_another_stream_without_workspace(dev):
    # Outputs and workspace allocated inside the call, which runs on a stream
    # of its own: the current stream's later allocations must not take them.
    _say("another stream")
    gen = _gen(15)
    X, dH = _normal((500, 300), gen, dev, torch.float16), _normal((500, 400), gen, dev, torch.float16)
    Wg, Wu = (_normal((400, 300), gen, dev, torch.float16, 0.1) for _ in range(2))
    P = torch.empty(500, 800, device=dev)
    sg.glu(X, Wg, Wu, preact=P)
    alone = sg.glu_backward(dH, X, Wg, Wu, P)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    for stream in (s, s.cuda_stream):
        for _ in range(3):
            got = sg.glu_backward(dH, X, Wg, Wu, P, stream=stream)
            junk = [torch.full((1 << 21,), float("nan"), dtype=torch.float16, device=dev) for _ in range(4)]
            w = sg.w4_quantize(Wg, 64, stream=stream)
            y = sg.w4_matmul(X, w, stream=stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, alone))
            assert torch.equal(y, sg.w4_matmul(X, sg.w4_quantize(Wg, 64)))
            del junk


def test_offsets_past_32_bits(dev):
    # Rows 256 MiB apart: offsets within one operand reach 10 GiB.
    M, F, K, S = 33, 40, 64, 1 << 27
    t = torch.bfloat16
    _say("far rows")
    big = torch.empty(F * S, dtype=t, device=dev)
    place = [0]

    def far(rows, cols, dtype=t):
        per = torch.empty(0, dtype=dtype).element_size() // 2
        v = big.view(dtype).as_strided((rows, cols), (S // per, 1), place[0] // per)
        place[0] += (cols * per + 63) // 64 * 64
        return v

    gen = _gen(16)
    near = [_ints(s, gen, -2, 2, dev, t) for s in ((M, K), (F, K), (F, K), (M, F))]
    X, Wg, Wu, dH = (far(*v.shape).copy_(v) for v in near)
    H, dX, dWg, dWu = far(M, F), far(M, K), far(F, K), far(F, K)
    P = far(M, 2 * F, torch.float32)
    sg.glu(X, Wg, Wu, "relu", out=H, preact=P)
    sg.glu_backward(dH, X, Wg, Wu, P, "relu", dX, dWg, dWu)
    p = torch.empty(M, 2 * F, device=dev)
    assert torch.equal(H, sg.glu(near[0], near[1], near[2], "relu", preact=p)) and torch.equal(P, p)
    for a, b in zip((dX, dWg, dWu), sg.glu_backward(near[3], near[0], near[1], near[2], p, "relu")):
        assert torch.equal(a, b)
    q = big.view(torch.uint8).as_strided((F, K // 2), (2 * S, 1), 2 * place[0])
    place[0] += 64
    w = sg.w4_quantize(Wg, 32)
    q.copy_(w.q)
    for rows in (1, M):
        y = far(rows, F)
        sg.w4_matmul(X[:rows], sg.W4(q, w.scales, None, K, 32), out=y)
        assert torch.equal(y, sg.w4_matmul(near[0][:rows], w))
    back = far(F, K)
    sg.w4_dequantize(sg.W4(q, w.scales, None, K, 32), out=back)
    assert torch.equal(back, sg.w4_dequantize(w))
