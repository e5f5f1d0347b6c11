"""The second parts of dG and dU in the gated block's backward pass, bit for bit:
whole-number inputs whose dG and dU have more bits than the type and whose
sums are exact in FP32 (ffn_parts.py), so that each gradient is the exact
value rounded once. A second part left out, negated or given to the other
matrix changes them (test_ffn_parts_cpu.py)."""
import pytest

torch = pytest.importorskip("torch")
import ffn_parts as parts  # noqa: E402
import ffn_ref as ref  # noqa: E402
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("t", parts.BITS, ids=str)
@pytest.mark.parametrize("case", parts.CASES, ids=str)
def test_second_parts(case, t, pad):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    print("[gpu] second parts", case, t, pad, flush=True)
    args = parts.inputs(case)
    want = parts.sums(*parts.kept(*args), *args[1:])
    dH, X, Wg, Wu = (ref.laid_out(v.to("cuda:0", t), pad, pad)[0] for v in args)
    P = torch.empty(X.shape[0], 2 * Wg.shape[0], device="cuda:0")
    sg.glu(X, Wg, Wu, "relu", preact=P)
    for name, a, b in zip(("dX", "dWg", "dWu"), sg.glu_backward(dH, X, Wg, Wu, P, "relu"), want):
        assert torch.equal(a.cpu(), b.to(t)), name
