"""Products of matrices in 8 bits and the gated block over them against 64-bit
references (i8_ref.py). With scales that are powers of two and sums below 2^24 a
result is the exact value rounded once, and compared for equality; others
within bounds that count each rounding. Operands sit in buffers padded with numbers
that no result may show, outputs in buffers whose surroundings have to stay as
they were."""
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


def _gen(*seed):
    g = torch.Generator()
    g.manual_seed(hash(seed) & 0xFFFFFFFF)
    return g


def _say(*a):
    print("[gpu]", *a, flush=True)


def _out(rows, cols, dtype, dev, layout):
    return ref.laid_out(torch.full((rows, cols), float("nan"), dtype=dtype, device=dev), *layout)


def _matrix(rows, K, gen, dev, most=127, layout=(0, 0), exact=True):
    """A matrix in 8 bits in a buffer of 113s, and a packed copy."""
    q = torch.randint(-most, most + 1, (rows, K), generator=gen).to(dev, torch.int8)
    s = 2.0 ** torch.randint(-3, 3, (rows,), generator=gen) if exact else torch.rand((rows,), generator=gen) + 1e-3
    s = s.to(dev, torch.float32)
    return sg.I8(ref.laid_out(q, *layout, fill=113)[0], s), sg.I8(q, s)


def _close(got, want, bound, what):
    d = (got.double() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((d / bound).nan_to_num(nan=1e30).max()):.3g} of its bound, first at "
                           f"{bad.nonzero()[0].tolist()}")


# (M, F, K): single elements, tails in each direction, rows of less than a 16-byte
# chunk, whole tiles and more than one tile of every kernel
SHAPES = [(1, 1, 1), (1, 7, 1000), (1, 300, 15), (2, 300, 16), (3, 65, 31), (5, 64, 64), (16, 96, 256), (17, 33, 65),
          (32, 130, 1040), (33, 64, 144), (64, 128, 128), (70, 31, 1025), (128, 64, 384), (129, 257, 383),
          (300, 200, 77), (257, 512, 128), (2, 9, 2), (4, 17, 3), (6, 40, 7), (12, 3800, 180), (9, 8200, 40),
          (2, 33, 4200), (1, 8200, 2064), (3, 4100, 1030), (7, 5000, 520), (40, 5, 3000), (100, 300, 13)]
LARGE = [(3000, 4136, 288), (2904, 72, 8400), (72, 2600, 5456), (520, 264, 400), (100, 3001, 260), (2500, 65, 134),
         (1201, 1203, 1205), (2050, 2048, 16), (600, 9000, 130), (4000, 4000, 100), (300, 2100, 9000),
         (500, 3100, 272), (2100, 1500, 272), (2100, 3100, 261), (1500, 5000, 1072), (2000, 2050, 1040), (130, 8200, 528),
         (3000, 8200, 525), (64, 4100, 1040), (64, 4100, 1051), (1000, 4100, 527), (260, 1030, 4112), (66, 5500, 272)]
LAYOUTS = [(0, 0), (16, 16), (3, 1)]


def _check(shape, dtype, layout, dev, seed):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    gen = _gen(seed, shape)
    most = 127 if K < 900 else 30        # sums below 2^24 are FP32 numbers
    (x, xp), (a, ap), (b, bp) = (_matrix(r, K, gen, dev, most, layout) for r in (M, F, F))
    y, flat = _out(M, F, t, dev, layout)
    assert sg.i8_matmul(x, a, out=y) is y
    torch.cuda.synchronize()
    g, u = i8_ref.product(xp, ap), i8_ref.product(xp, bp)
    assert torch.equal(y, g.to(t)) and ref.around_untouched(flat, y)
    h, flat = _out(M, F, t, dev, layout)
    sg.i8_glu(x, a, b, "relu", out=h)
    torch.cuda.synchronize()
    # G and U are exact FP32 numbers; their product is rounded to FP32 and to the type
    assert torch.equal(h, (g.clamp(min=0).float() * u.float()).to(t)) and ref.around_untouched(flat, h)


@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_products(dev, shape, dtype, layout):
    _say("i8 products", shape, dtype, layout)
    _check(shape, dtype, layout, dev, 1)


@pytest.mark.parametrize("layout", LAYOUTS[:2], ids=str)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", LARGE, ids=lambda s: "x".join(map(str, s)))
def test_large_products(dev, shape, dtype, layout):
    _say("i8 large products", shape, dtype, layout)
    _check(shape, dtype, layout, dev, 2)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ref.DTYPES)
@pytest.mark.parametrize("shape", [(1, 64, 256), (9, 130, 77), (50, 700, 520), (300, 400, 300)], ids=str)
def test_random_scales(dev, shape, dtype, act):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    _say("i8 random", shape, dtype, act)
    gen = _gen(3, shape)
    x, a, b = (_matrix(r, K, gen, dev, exact=False)[1] for r in (M, F, F))
    x = sg.I8(x.q, x.scales * (4.0 / 127 / 73 * K ** -0.5))
    want = i8_ref.product(x, a)
    _close(sg.i8_matmul(x, a, t), want, i8_ref.product_bound(want, dtype), "Y")
    _close(sg.i8_glu(x, a, b, act, t), i8_ref.glu(x, a, b, act), i8_ref.glu_bound(x, a, b, act, dtype), act)


@pytest.mark.parametrize("M", [1, 3, 7, 20, 60, 200])
def test_a_products_kernel_does_not_show(dev, M):
    # Sums are exact, so a row's results do not depend on the rows beside it.
    _say("rows apart", M)
    gen = _gen(4)
    x, a, b = (_matrix(r, 1111, gen, dev, exact=False)[1] for r in (300, 500, 500))
    for t in ref.DTYPES.values():
        y, h = sg.i8_matmul(x, a, t), sg.i8_glu(x, a, b, "gelu_tanh", t)
        part = sg.I8(x.q[:M], x.scales[:M])
        assert torch.equal(sg.i8_matmul(part, a, t), y[:M]) and torch.equal(sg.i8_glu(part, a, b, "gelu_tanh", t), h[:M])


@pytest.mark.parametrize("M", [1, 4, 20, 70])
def test_the_longest_sums(dev, M):
    # 131071 products of -128 and -128: 2^31 - 2^14, the largest; and the smallest, of -128 and 127.
    _say("longest sums", M)
    K = 131071
    x = sg.I8(torch.full((M, K), -128, dtype=torch.int8, device=dev), torch.ones(M, device=dev))
    w = sg.I8(torch.full((3, K), -128, dtype=torch.int8, device=dev), torch.ones(3, device=dev))
    w.q[1] = 127
    w.q[2, ::2] = 127
    y = sg.i8_matmul(x, w)
    want = x.q.double() @ w.q.double().T
    assert float(want.max()) == 131071 * 16384 and torch.equal(y, want.float())
    h = sg.i8_glu(x, w, sg.I8(w.q, torch.full((3,), 2.0 ** -40, device=dev)), "relu")
    assert torch.equal(h, (want.clamp(min=0).float() * (want.float() * 2.0 ** -40)))


@pytest.mark.parametrize("M", [1, 4, 20, 70])
def test_scales_that_are_not_ordinary(dev, M):
    # Products of scales that leave FP32's range while the results do not; zeros,
    # infinities and NaN stay in their rows and columns.
    _say("scales not ordinary", M)
    gen = _gen(5)
    F, K = 90, 200
    x, w = (_matrix(r, K, gen, dev, 127)[1] for r in (M, F))
    sx, sw = x.scales, w.scales
    for i, j in ((2.0 ** -120, 2.0 ** 110), (2.0 ** 120, 2.0 ** -130), (2.0 ** -149, 2.0 ** 127), (2.0 ** 127, 2.0 ** -149)):
        want = i8_ref.product((x.q, sx * 0 + i), (w.q, sw * 0 + j))
        assert torch.equal(sg.i8_matmul(sg.I8(x.q, sx * 0 + i), sg.I8(w.q, sw * 0 + j)), want.float())
    bad = sw.clone()
    bad[3], bad[5], bad[7] = 0.0, float("inf"), float("nan")
    y = sg.i8_matmul(x, sg.I8(w.q, bad))
    sums = x.q.double() @ w.q.double().T
    assert (y[:, 3] == 0).all() and y[:, 7].isnan().all()
    assert torch.equal(y[:, 5].isnan(), sums[:, 5] == 0) and torch.equal(y[:, 5] == float("inf"), sums[:, 5] > 0)
    rest = torch.ones(F, dtype=torch.bool, device=dev)
    rest[[3, 5, 7]] = False
    plain = sg.i8_matmul(x, w)
    assert torch.equal(y[:, rest], plain[:, rest])
    h = sg.i8_glu(x, sg.I8(w.q, bad), w)
    assert torch.equal(h[:, rest], sg.i8_glu(x, w, w)[:, rest]) and h[:, 7].isnan().all()
    if M > 1:
        badx = sx.clone()
        badx[1] = float("nan")
        y = sg.i8_matmul(sg.I8(x.q, badx), w)
        keep = torch.arange(M, device=dev) != 1
        assert y[1].isnan().all() and torch.equal(y[keep], plain[keep])


@pytest.mark.parametrize("act", ref.ACTS)
def test_glu_far_arguments(dev, act):
    # G from -200 to 200; U is 1, so H is act(G).
    _say("i8_glu far", act)
    n = torch.tensor([-100, -90, -60, -30, -10, -1, 0, 1, 10, 45, 90, 127], device=dev)
    x = sg.I8(torch.stack((n, torch.ones_like(n)), 1).to(torch.int8).contiguous(), torch.ones(12, device=dev))
    g = sg.I8(torch.tensor([[1, 0]], dtype=torch.int8, device=dev), torch.tensor([2.0], device=dev))
    u = sg.I8(torch.tensor([[0, 1]], dtype=torch.int8, device=dev), torch.tensor([1.0], device=dev))
    for name, t in ref.DTYPES.items():
        _close(sg.i8_glu(x, g, u, act, t), i8_ref.glu(x, g, u, act), i8_ref.glu_bound(x, g, u, act, name), act)


def test_empty_sums(dev):
    _say("i8 empty sums")
    nan = float("nan")
    e = lambda r, c: torch.empty(r, c, dtype=torch.int8, device=dev)   # noqa: E731
    s = lambda n: torch.full((n,), nan, device=dev)                    # noqa: E731
    for t in ref.DTYPES.values():
        x, w = sg.I8(e(3, 0), s(3)), sg.I8(e(5, 0), s(5))
        out = torch.full((3, 5), nan, dtype=t, device=dev)
        assert (sg.i8_matmul(x, w, out=out) == 0).all()
        out.fill_(nan)
        assert (sg.i8_glu(x, w, w, out=out) == 0).all()
        assert sg.i8_matmul(sg.I8(e(0, 4), s(0)), sg.I8(e(5, 4), s(5)), t).shape == (0, 5)
        assert sg.i8_matmul(sg.I8(e(3, 4), s(3)), sg.I8(e(0, 4), s(0)), t).shape == (3, 0)


def test_offsets_past_32_bits(dev):
    # Rows 2^31 bytes and more apart, in X, W and Y.
    _say("i8 far rows")
    gen = _gen(6)
    K, ld = 300, (1 << 31) + 64
    for M in (1, 3, 40, 70):
        x, a, b = (_matrix(r, K, gen, dev, exact=False)[1] for r in (M, 3, 3))
        fa, fb = (torch.empty(2 * ld + K, dtype=torch.int8, device=dev).as_strided((3, K), (ld, 1)) for _ in range(2))
        fa.copy_(a.q)
        fb.copy_(b.q)
        assert torch.equal(sg.i8_matmul(x, sg.I8(fa, a.scales)), sg.i8_matmul(x, a))
        assert torch.equal(sg.i8_glu(x, sg.I8(fa, a.scales), sg.I8(fb, b.scales)), sg.i8_glu(x, a, b))
        # and the other way round: three far tokens
        y = torch.empty(2 * ld + M, dtype=torch.float16, device=dev).as_strided((3, M), (ld, 1))
        assert torch.equal(sg.i8_matmul(sg.I8(fa, a.scales), x, out=y), sg.i8_matmul(a, x, torch.float16))
        del fa, fb, y


def test_more_rows_of_blocks_than_a_second_grid_extent(dev):
    # 65537 blocks of 64 rows of few features and a long sum, where the rows' kernel would be the fastest.
    _say("i8 four million rows")
    M, F, K = 65536 * 64 + 1, 16, 10240
    if torch.cuda.mem_get_info(dev)[0] < 48 << 30:
        pytest.skip("less than 48 GiB of memory free")
    gen = _gen(7)
    rows = torch.tensor([0, 1, 63, 64, 65535 * 64 - 1, 65535 * 64, M - 2, M - 1], device=dev)
    _, some = _matrix(len(rows), K, gen, dev)
    _, w = _matrix(F, K, gen, dev)
    q, scales = torch.zeros(M, K, dtype=torch.int8, device=dev), torch.ones(M, device=dev)
    q[rows], scales[rows] = some.q, some.scales
    got = sg.i8_matmul(sg.I8(q, scales), w)
    assert torch.equal(got[rows], sg.i8_matmul(some, w))
    got[rows] = 0
    assert (got == 0).all()
    del q
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# As they are used together
# ---------------------------------------------------------------------------
def _block(X, R, Wn, wg, wu, wd, act, t):
    """norm to 8 bits, gated block, its result to 8 bits, second product: the
    feed-forward half of a layer; returns (its output, the residual stream)."""
    H = torch.empty_like(X)
    x = sg.rms_norm_i8(X, Wn, 1e-5, residual=R, total=H)
    h = sg.i8_quantize(sg.i8_glu(x, wg, wu, act, t))
    return sg.i8_matmul(h, wd, t), H


@pytest.mark.parametrize("M", [1, 5, 33, 300])
@pytest.mark.parametrize("dtype", ref.DTYPES)
def test_a_feed_forward_block(dev, dtype, M):
    t = ref.DTYPES[dtype]
    _say("i8 block", dtype, M)
    gen = _gen(7, M)
    K, F = 520, 1100
    X, R = (torch.randn((M, K), generator=gen, dtype=torch.float64).to(dev, t) for _ in range(2))
    Wn = (1 + 0.2 * torch.randn(K, generator=gen, dtype=torch.float64)).to(dev, t)
    wg, wu, wd = (sg.i8_quantize((torch.randn(s, generator=gen, dtype=torch.float64) * s[1] ** -0.5).to(dev, t))
                  for s in ((F, K), (F, K), (K, F)))
    y, H = _block(X, R, Wn, wg, wu, wd, "silu", t)
    # the same chain by the definitions, from the stored numbers of each step
    assert torch.equal(H, i8_ref.total(X, R))
    x = sg.rms_norm_i8(X, Wn, 1e-5, residual=R)
    q, top = i8_ref.levels(H.double() * Wn.double())
    assert (x.q.int() - q.int()).abs().max() <= (1 if dtype == "f32" else 0)
    h = sg.i8_glu(x, wg, wu, "silu", t)
    _close(h, i8_ref.glu(x, wg, wu, "silu"), i8_ref.glu_bound(x, wg, wu, "silu", dtype), "H")
    p = sg.i8_quantize(h)
    assert torch.equal(p.q, i8_ref.levels(h)[0])
    want = i8_ref.product(p, wd)
    _close(y, want, i8_ref.product_bound(want, dtype), "Y")
    # and near what the block without 8 bits gives: three roundings to 1/254 of a row's largest
    # number, each a relative error of some 0.5% of a row's norm
    n = i8_ref.norm(H, Wn, 1e-5)
    a, b, c = (sg.i8_dequantize(w).double() for w in (wg, wu, wd))
    full = (torch.nn.functional.silu(n @ a.T) * (n @ b.T)) @ c.T
    assert (y.double() - full).norm() / full.norm() < 0.04


@pytest.mark.parametrize("M", [1, 20, 300])
def test_a_block_in_a_replayed_graph(dev, M):
    # Two blocks captured once; new inputs before each replay, eager work and
    # synchronizations between them, every replay checked.
    _say("i8 graph", M)
    t = torch.bfloat16
    gen = _gen(8, M)
    K, F = 512, 1024
    X, R = (torch.randn((M, K), generator=gen).to(dev, t) for _ in range(2))
    Wn = torch.ones(K, dtype=t, device=dev)
    wg, wu, wd = (sg.i8_quantize(torch.randn(s, generator=gen).to(dev, t)) for s in ((F, K), (F, K), (K, F)))
    dY = torch.randn((M, K), generator=gen).to(dev, t)

    def work():
        y, H = _block(X, R, Wn, wg, wu, wd, "gelu", t)
        z, H2 = _block(y, H, Wn, wg, wu, wd, "silu", t)
        r = torch.empty(M, device=dev)
        o = sg.rms_norm(z, Wn, residual=H2, total=H2, rstd=r)
        return [z, o, *sg.rms_norm_backward(dY, H2, Wn, r)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = work()
    for i in range(4):
        X.copy_(torch.randn((M, K), generator=gen).to(dev, t))
        R.mul_(0.5)
        want = [v.clone() for v in work()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_the_same_bits_each_time(dev):
    _say("i8 repeated")
    gen = _gen(9)
    X, dY = (torch.randn((700, 1030), generator=gen).to(dev) for _ in range(2))
    W = torch.ones(1030, device=dev)
    r = torch.empty(700, device=dev)
    first = None
    for _ in range(5):
        y = sg.rms_norm(X, W, rstd=r)
        now = [y, *sg.rms_norm_backward(dY, X, W, r), *sg.rms_norm_i8(X, W)]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.fixture(scope="module")
def job(dev):
    gen = _gen(10)
    t = torch.bfloat16
    X, R, dY = (torch.randn((300, 256), generator=gen).to(dev, t) for _ in range(3))
    W = torch.ones(256, dtype=t, device=dev)
    r = torch.empty(300, device=dev)
    sg.rms_norm(X, W, rstd=r)
    x = sg.i8_quantize(X)
    a, b = (sg.i8_quantize(torch.randn((512, 256), generator=gen).to(dev, t)) for _ in range(2))
    torch.cuda.synchronize()
    slow = torch.zeros(1 << 28, device=dev)                      # 1 GiB: a pass takes 0.4 ms
    calls = {
        "rms_norm": lambda s: [sg.rms_norm(X, W, residual=R, stream=s)],
        "rms_norm_backward": lambda s: list(sg.rms_norm_backward(dY, X, W, r, stream=s)),
        "rms_norm_i8": lambda s: list(sg.rms_norm_i8(X, W, residual=R, stream=s)),
        "i8_quantize": lambda s: list(sg.i8_quantize(X, stream=s)),
        "i8_dequantize": lambda s: [sg.i8_dequantize(x, stream=s)],
        "i8_matmul": lambda s: [sg.i8_matmul(x, a, t, stream=s)],
        "i8_glu": lambda s: [sg.i8_glu(x, a, b, dtype=t, stream=s)],
    }
    return calls, slow, sg.rms_norm_backward_workspace(X)


CALLS = ["rms_norm", "rms_norm_backward", "rms_norm_i8", "i8_quantize", "i8_dequantize", "i8_matmul", "i8_glu"]


@pytest.mark.parametrize("address", [False, True], ids=["stream", "address"])
@pytest.mark.parametrize("name", CALLS)
def test_memory_still_in_use_is_not_taken(dev, job, name, address):
    calls, slow, workspace = job
    call = calls[name]
    _say("memory in use", name, address)
    alone = call(None)
    sizes = [v.numel() * v.element_size() for v in alone] + [workspace]
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    for _ in range(3):
        held = [torch.full((n,), i + 1, dtype=torch.uint8, device=dev) for i, n in enumerate(sizes)]
        torch.cuda.synchronize()
        for _ in range(10):
            slow.add_(1)
        copies = [h.clone() for h in held]
        del held
        got = call(s.cuda_stream if address else s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone))
        torch.cuda.synchronize()
        for i, c in enumerate(copies):
            assert (c == i + 1).all()


def test_calls_on_two_streams_at_once(dev, job):
    calls, slow, _ = job
    _say("two streams")
    alone = {n: [v.clone() for v in calls[n](None)] for n in CALLS}
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
    for _ in range(3):
        got = [(n, calls[n](s)) for n in CALLS for s in (a, b)]
        torch.cuda.synchronize()
        for n, g in got:
            assert all(torch.equal(v, w) for v, w in zip(g, alone[n])), n
