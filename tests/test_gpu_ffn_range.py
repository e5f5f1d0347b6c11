"""The gradients of the gated block where dG and dU do not fit half as they are:
large ones whose gradients are ordinary numbers, small ones, rows of different
sizes, and rows that hold an infinity or NaN (64-bit references, ffn_ref.py)."""
import pytest

torch = pytest.importorskip("torch")
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu
HALF = torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _normal(shape, gen, dev, scale):
    return (torch.randn(shape, generator=gen, dtype=torch.float64) * scale).to(dev, HALF)


def _step(dH, X, Wg, Wu, act="silu"):
    P = torch.empty(X.shape[0], 2 * Wg.shape[0], device=X.device)
    sg.glu(X, Wg, Wu, act, preact=P)
    ws = torch.full((sg.glu_backward_workspace(X, Wg.shape[0]),), 0xFF, dtype=torch.uint8, device=X.device)
    return sg.glu_backward(dH, X, Wg, Wu, P, act, workspace=ws)


def _bounds(dH, X, Wg, Wu, act):
    """Elementwise bounds of dX, dWg and dWu. What is kept of dG and dU is off
    by half a step (where it is in two parts, by half a step of half a step) or
    by 2^-40 of the largest of them, and by its evaluation in FP32 (as in
    ffn_ref.glu_grads_bounds); the products are exact, summed in FP32 and
    rounded once."""
    r, t = ref.HALF_STEP["f16"], ref.TINY["f16"]
    rd = r * r if dH.numel() <= 16384 else r
    g, u = X @ Wg.T, X @ Wu.T
    e = ref.sum_error(X.shape[1])
    eg, eu = e * (X.abs() @ Wg.abs().T), e * (X.abs() @ Wu.abs().T)
    a, s = ref.act(g, act)
    h, ev = dH.abs(), ref.act_eval_error(g, act)
    edg = h * ((u.abs() + eu) * (eg + (s.abs() + 1.2) * (ev + 2.0 ** -22)) + s.abs() * eu)
    edu = h * (1.13 * eg + a.abs() * (ev + 2.0 ** -23))
    dg, du = dH * u * s, dH * a
    least = 2.0 ** -40 * 2 * max(float(dg.abs().max()), float(du.abs().max()))   # (doubled: evaluated in FP32)
    edg = edg + rd * (dg.abs() + edg) + least
    edu = edu + rd * (du.abs() + edu) + least

    M, F = dH.shape
    mags = (dg.abs() @ Wg.abs() + du.abs() @ Wu.abs(), dg.abs().T @ X.abs(), du.abs().T @ X.abs())
    errs = (edg @ Wg.abs() + edu @ Wu.abs(), edg.T @ X.abs(), edu.T @ X.abs())
    # the last rounding is of the result itself, not of its magnitudes
    exact = (dg @ Wg + du @ Wu, dg.T @ X, du.T @ X)
    return [(x, err + ref.sum_error(n) * (mag + err) + r * (x.abs() + 2 * err) + t)
            for x, mag, err, n in zip(exact, mags, errs, (2 * F, M, M))]


# scales of (X, Wg, Wu, dH); Wg and Wu also by K^-0.5
KINDS = {"large": (2.0 ** -8, 2.0 ** -4, 2.0 ** 14, 8000.0),   # U of tens: dG to a million, G near 0, gradients of thousands
         "small": (1.0, 1.0, 0.01, 5e-5), "tiny": (1.0, 1.0, 0.01, 1e-5)}


@pytest.mark.parametrize("act", ref.ACTS[:3])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(256, 256, 256), (9, 130, 77), (40, 33, 50), (300, 1000, 511), (2500, 72, 264),
                                   (1, 3000, 6)], ids=str)
def test_gradients_keep_their_range(dev, shape, kind, act):
    M, F, K = shape
    print("[gpu] half range", shape, kind, act, flush=True)
    x, wg, wu, h = KINDS[kind]
    gen = _gen(31)
    X, dH = _normal((M, K), gen, dev, x), _normal((M, F), gen, dev, h)
    Wg, Wu = (_normal((F, K), gen, dev, w * K ** -0.5) for w in (wg, wu))
    got = _step(dH, X, Wg, Wu, act)
    for name, a, (b, bound) in zip(("dX", "dWg", "dWu"), got, _bounds(*(v.double() for v in (dH, X, Wg, Wu)), act)):
        fits = b.abs() < 65000   # (the rest, in "large" where sums are long, may round to an infinity)
        assert fits.any()
        d = (a.double() - b).abs()
        assert (d <= bound)[fits].all(), f"{name}: worst {float((d / bound)[fits].nan_to_num(nan=1e30).max()):.3g} of its bound"


def test_rows_of_different_sizes(dev):
    # One row's gradients 2^22 times the others': each row of dX within its bound.
    print("[gpu] half rows", flush=True)
    gen = _gen(32)
    M, F, K = 130, 200, 96
    X, dH = _normal((M, K), gen, dev, 1.0), _normal((M, F), gen, dev, 2.0 ** -8)
    dH[7] = dH[7] * 2.0 ** 22
    Wg, Wu = (_normal((F, K), gen, dev, K ** -0.5) for _ in range(2))
    dX = _step(dH, X, Wg, Wu)[0].double()
    want, bound = _bounds(*(v.double() for v in (dH, X, Wg, Wu)), "silu")[0]
    assert ((dX - want).abs() <= bound).all()
    rest = [m for m in range(M) if m != 7]
    # (in the norm: half a step of what is kept and of the result, and 2^-40 of 2^16 where
    # the others' values are 2^-8: 2^-16 of them)
    err = (dX - want)[rest].norm() / want[rest].norm()
    assert float(err) <= 2 * ref.HALF_STEP["f16"] + 2.0 ** -13


@pytest.mark.parametrize("shape", [(70, 100, 64), (200, 256, 128)], ids=str)
def test_infinities_stay_in_their_rows(dev, shape):
    M, F, K = shape
    print("[gpu] half infinities", shape, flush=True)
    gen = _gen(33)
    X, dH = _normal((M, K), gen, dev, 1.0), _normal((M, F), gen, dev, 1.0)
    Wg, Wu = (_normal((F, K), gen, dev, K ** -0.5) for _ in range(2))
    dH[3] = 0
    dH[5] = 0
    clean = _step(dH, X, Wg, Wu)
    dH[3, 10] = float("inf")
    dH[5, 20] = float("nan")
    got = _step(dH, X, Wg, Wu)
    rows = [m for m in range(M) if m not in (3, 5)]
    feats = [f for f in range(F) if f not in (10, 20)]
    assert not torch.isfinite(got[0][3]).any() and torch.isnan(got[0][5]).all()
    assert torch.equal(got[0][rows], clean[0][rows])
    for a, b in zip(got[1:], clean[1:]):
        assert torch.equal(a[feats], b[feats]) and torch.isnan(a[20]).all() and not torch.isfinite(a[10]).any()


def test_no_gradient_is_zero(dev):
    gen = _gen(34)
    X = _normal((50, 40), gen, dev, 1.0)
    Wg, Wu = (_normal((60, 40), gen, dev, 0.2) for _ in range(2))
    for g in _step(torch.zeros(50, 60, dtype=HALF, device=dev), X, Wg, Wu):
        assert (g == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_many_workgroups_find_the_largest(dev, kind):
    # More values than one pass of all workgroups that look for the largest takes;
    # it is the last one.
    M, F, K = 1500, 1500, 40
    print("[gpu] half, many workgroups", kind, flush=True)
    x, wg, wu, h = KINDS[kind]
    gen = _gen(35)
    X, dH = _normal((M, K), gen, dev, x), _normal((M, F), gen, dev, h / 8)
    Wg, Wu = (_normal((F, K), gen, dev, w * K ** -0.5) for w in (wg, wu))
    dH[-1, -1] = h * 4
    for name, a, (b, bound) in zip(("dX", "dWg", "dWu"), _step(dH, X, Wg, Wu),
                                   _bounds(*(v.double() for v in (dH, X, Wg, Wu)), "silu")):
        fits = b.abs() < 65000
        d = (a.double() - b).abs()
        assert fits.any() and (d <= bound)[fits].all(), name


def test_a_graph_follows_its_inputs(dev):
    # One captured step, replayed on gradients of other sizes: each replay scales
    # by what it finds.
    print("[gpu] half graph", flush=True)
    gen = _gen(36)
    M, F, K = 150, 260, 72
    X, base = _normal((M, K), gen, dev, 1.0), _normal((M, F), gen, dev, 1.0)
    Wg, Wu = (_normal((F, K), gen, dev, K ** -0.5) for _ in range(2))
    dH = base.clone()
    P = torch.empty(M, 2 * F, device=dev)
    outs = [torch.empty(r, K, dtype=HALF, device=dev) for r in (M, F, F)]
    ws = torch.empty(sg.glu_backward_workspace(X, F), dtype=torch.uint8, device=dev)

    def step():
        sg.glu(X, Wg, Wu, preact=P)
        sg.glu_backward(dH, X, Wg, Wu, P, dX=outs[0], dWg=outs[1], dWu=outs[2], workspace=ws)

    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for scale in (1.0, 2.0 ** -14, 2.0 ** 9, 0.0, 2.0 ** -20, 1.0):
        dH.copy_(base * scale)
        want = _step(dH.clone(), X, Wg, Wu)
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), scale
    del g


def test_one_workspace_for_calls_of_other_sizes(dev):
    print("[gpu] half, one workspace", flush=True)
    gen = _gen(37)
    jobs = []
    for M, F, K, h in ((300, 500, 64, 1e-4), (20, 40, 96, 5000.0), (500, 300, 33, 1.0)):
        X, dH = _normal((M, K), gen, dev, 0.1), _normal((M, F), gen, dev, h)
        Wg, Wu = (_normal((F, K), gen, dev, K ** -0.5) for _ in range(2))
        P = torch.empty(M, 2 * F, device=dev)
        sg.glu(X, Wg, Wu, preact=P)
        jobs.append((dH, X, Wg, Wu, P))
    ws = torch.empty(max(sg.glu_backward_workspace(j[1], j[2].shape[0]) for j in jobs), dtype=torch.uint8, device=dev)
    alone = [sg.glu_backward(*j) for j in jobs]
    for _ in range(2):
        got = [sg.glu_backward(*j, workspace=ws) for j in jobs]
        assert all(torch.equal(a, b) for x, y in zip(got, alone) for a, b in zip(x, y))
