"""FP32 gradients of rows so far apart that a slice of them spans more than
31-bit offsets."""
import pytest

torch = pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1300, 1301])
def test_far_rows_of_the_activations(K):
    # More tiles than the operators' own kernels take by themselves (640 of 64 x 64).
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    dev = torch.device("cuda:0")
    M, F, S = 40, 1300, 1 << 25
    print("[gpu] far rows f32", K, flush=True)
    gen = torch.Generator().manual_seed(51)
    ints = lambda *s: torch.randint(-2, 3, s, generator=gen).to(dev, torch.float32)   # noqa: E731
    near, dH, Wg, Wu = ints(M, K), ints(M, F), ints(F, K), ints(F, K)
    X = torch.empty(M * S, device=dev).as_strided((M, K), (S, 1)).copy_(near)
    P, p = (torch.empty(M, 2 * F, device=dev) for _ in range(2))
    assert torch.equal(sg.glu(X, Wg, Wu, "relu", preact=P), sg.glu(near, Wg, Wu, "relu", preact=p))
    assert torch.equal(P, p)
    x, wg, wu, dh = (v.double() for v in (near, Wg, Wu, dH))
    g, u = x @ wg.T, x @ wu.T
    dg, du = dh * u * (g > 0), dh * g.clamp(min=0)
    want = (dg @ wg + du @ wu, dg.T @ x, du.T @ x)       # whole numbers below 2^24: exact in FP32
    assert max(float(v.abs().max()) for v in want) < 2 ** 24
    for name, a, b in zip(("dX", "dWg", "dWu"), sg.glu_backward(dH, X, Wg, Wu, P, "relu"), want):
        assert torch.equal(a.double(), b), name


@pytest.mark.parametrize("K", [1300, 1301])
def test_far_rows_of_the_weights(K):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    dev = torch.device("cuda:0")
    M, F, S = 1300, 40, 1 << 25
    print("[gpu] far weights f32", K, flush=True)
    gen = torch.Generator().manual_seed(52)
    ints = lambda *s: torch.randint(-2, 3, s, generator=gen).to(dev, torch.float32)   # noqa: E731
    X, dH, near = ints(M, K), ints(M, F), (ints(F, K), ints(F, K))
    buffer = torch.empty(F * S, device=dev)
    far = [buffer.as_strided((F, K), (S, 1), i * 4096).copy_(v) for i, v in enumerate(near)]
    outs = [buffer.as_strided((F, K), (S, 1), i * 4096) for i in (2, 3)]
    P, p = (torch.empty(M, 2 * F, device=dev) for _ in range(2))
    assert torch.equal(sg.glu(X, *far, "relu", preact=P), sg.glu(X, *near, "relu", preact=p)) and torch.equal(P, p)
    x, wg, wu, dh = (v.double() for v in (X, *near, dH))
    g, u = x @ wg.T, x @ wu.T
    dg, du = dh * u * (g > 0), dh * g.clamp(min=0)
    want = (dg @ wg + du @ wu, dg.T @ x, du.T @ x)
    assert max(float(v.abs().max()) for v in want) < 2 ** 24
    for name, a, b in zip(("dX", "dWg", "dWu"), sg.glu_backward(dH, X, *far, P, "relu", dWg=outs[0], dWu=outs[1]), want):
        assert torch.equal(a.double(), b), name


@pytest.mark.parametrize("ld", [1 << 60, 1 << 40, (1 << 60) + 7])
@pytest.mark.parametrize("dtype,F", [(1, 20000), (2, 20000), (0, 20000), (0, 64), (1, 64)])
def test_any_leading_dimension_of_a_single_row(dtype, F, ld):
    # One row of X, so its leading dimension is of no consequence. An infinity in it
    # shows if the row is read for others: those, times zero, would make it NaN.
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    dev = torch.device("cuda:0")
    print("[gpu] one row", dtype, F, ld, flush=True)
    t = (torch.float32, torch.bfloat16, torch.float16)[dtype]
    K = 64
    X = torch.arange(1, K + 1, device=dev).to(t)[None]
    two_parts = dtype != 0 and F <= 16384          # (an infinity times a second part of zero is NaN)
    if not two_parts:
        X[0, 3] = float("inf")
    P = torch.ones(1, 2 * F, device=dev)           # G = U = 1: dG = dU = dH
    dH = torch.ones(1, F, dtype=t, device=dev)
    dWg, dWu = (torch.full((F, K), float("nan"), dtype=t, device=dev) for _ in range(2))
    need = sg.glu_backward_workspace(X, F)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    rc = sg.sgemm_f32_glu_bwd(dtype, 3, 1, F, K, X, ld, 0, K, 0, K, P, ld, dH, ld, 0, K, dWg, K, dWu, K, ws, need)
    torch.cuda.synchronize()
    assert rc == 0 and torch.equal(dWg, X.expand(F, K)) and torch.equal(dWu, X.expand(F, K))
    H = torch.full((1, F), float("nan"), dtype=t, device=dev)
    W = torch.ones(F, K, dtype=t, device=dev)
    assert sg.sgemm_f32_glu(dtype, 3, 1, F, K, X, ld, W, K, W, K, H, ld, None, 1) == 0
    torch.cuda.synchronize()
    g = X.double().sum()
    assert torch.equal(H, (g * g).to(t).expand(1, F))
