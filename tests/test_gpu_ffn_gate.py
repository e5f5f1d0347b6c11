"""The gate of 16-bit calls far from zero, where act(g) is small: it keeps its
relative error down to the type's smallest normal numbers, in every forward
kernel and in the gradients (64-bit references, ffn_ref.py)."""
import pytest

torch = pytest.importorskip("torch")
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu
FAR = [-200.0, -120.0, -103.0, -95.0, -92.0, -91.0, -90.5, -90.0, -89.0, -88.0, -87.5, -87.0, -60.0, -30.0, -17.0, -8.0, -3.0,
       -0.5, 0.0, 0.5, 3.0, 17.0, 90.0, 200.0]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")


def _inputs(M, F, K, t, dev):
    """G = FAR, one after the other along the rows, and U = 1, exactly."""
    X = torch.zeros(M, K, dtype=t, device=dev)
    X[:, 0] = torch.tensor(FAR, device=dev).repeat(-(-M // len(FAR)))[:M].to(t)
    X[:, 1] = 1
    Wg, Wu = (torch.zeros(F, K, dtype=t, device=dev) for _ in range(2))
    Wg[:, 0] = 1
    Wu[:, 1] = 1
    return X, Wg, Wu


# one row and few (vector units), rows that split K, tiles of both fills
@pytest.mark.parametrize("shape", [(1, 64, 64), (24, 10, 96), (24, 9000, 64), (300, 5000, 64), (300, 5000, 70)], ids=str)
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_far_gate(dev, dtype, act, shape):
    M, F, K = shape
    t = ref.DTYPES[dtype]
    print("[gpu] far gate", dtype, act, shape, flush=True)
    for at in range(len(FAR) if M == 1 else 1):
        X, Wg, Wu = _inputs(M, F, K, t, dev)
        if M == 1:
            X[0, 0] = FAR[at]
        g = X[:, :1].double().expand(M, F)
        want = ref.act(g, act)[0]
        H = sg.glu(X, Wg, Wu, act)
        # evaluation, one rounding, and a step of FP32's and the type's subnormals
        bound = want.abs() * (ref.act_eval_error(g, act) + ref.HALF_STEP[dtype] * 1.01) + ref.TINY[dtype]
        assert ((H.double() - want).abs() <= bound).all()
        if act == "silu" and dtype == "bf16":
            low = (g > -90.8) & (g < -87)
            assert (H[low] < -2.0 ** -126).all()       # normal numbers, not zero


@pytest.mark.parametrize("act", ref.ACTS[:3])
def test_far_gradients(dev, act):
    # bfloat16, one feature: dX[:, 0] = dH act'(g) and dX[:, 1] = dH act(g), each
    # from one product with 1, dG and dU in two parts.
    X, Wg, Wu = _inputs(len(FAR), 1, 16, torch.bfloat16, dev)
    dH = torch.ones(len(FAR), 1, dtype=torch.bfloat16, device=dev)
    print("[gpu] far gradients", act, flush=True)
    P = torch.empty(len(FAR), 2, device=dev)
    sg.glu(X, Wg, Wu, act, preact=P)
    dX = sg.glu_backward(dH, X, Wg, Wu, P, act)[0].double()
    g = X[:, 0].double()
    a, s = ref.act(g, act)
    e = ref.act_eval_error(g, act)
    for got, want, size in ((dX[:, 0], s, s.abs() + (g * s).abs()), (dX[:, 1], a, a.abs())):
        assert ((got - want).abs() <= size * (e + 2.0 ** -22) + want.abs() * 2.0 ** -8 * 1.01 + 2.0 ** -133).all()


def test_far_gate_of_4_bit_weights(dev):
    # A group's scale times (15 - 8) = 7 and the activations in sevenths: G = FAR
    # to a rounding of the input, U = 7.
    print("[gpu] far gate, 4 bits", flush=True)
    t = torch.bfloat16
    for M in (1, 2, len(FAR)):
        for first in range(0, len(FAR), M):
            X = torch.zeros(M, 64, dtype=t, device=dev)
            X[:, 0] = (torch.tensor(FAR[first:first + M], device=dev) / 7).to(t)
            X[:, 1] = 1
            q = torch.full((48, 64), 8, dtype=torch.uint8, device=dev)
            qg, qu = q.clone(), q.clone()
            qg[:, 0] = 15
            qu[:, 1] = 15
            ones = torch.ones(48, 2, dtype=t, device=dev)
            wg, wu = (sg.W4(v[:, 0::2] | (v[:, 1::2] << 4), ones, None, 64, 32) for v in (qg, qu))
            g = (7 * X[:, :1].double()).expand(M, 48)
            want = 7 * ref.act(g, "silu")[0]
            # G is summed as 31 x - 24 x and U as 31 - 24, in FP32: off by (31 + 24) 2^-22 |x| / |G|
            eg = 2.0 ** -22 * 8 * g.abs()
            bound = want.abs() * (ref.act_eval_error(g, "silu") + 2 * eg + 2.0 ** -8 * 1.01) + ref.TINY["bf16"]
            assert ((sg.w4_glu(X, wg, wu, "silu").double() - want).abs() <= bound).all()
