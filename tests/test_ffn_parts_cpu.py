"""That the inputs of ffn_parts.py show a mistake in the second parts of dG and
dU: the mistake is planted in the 64-bit form, on the CPU."""
import pytest

torch = pytest.importorskip("torch")
import ffn_parts as parts  # noqa: E402


@pytest.mark.parametrize("case", parts.CASES, ids=str)
def test_sums_are_exact(case):
    dH, X, Wg, Wu = parts.inputs(case)
    dg, du = parts.kept(dH, X, Wg, Wu)
    assert dH.numel() <= 16384
    assert max(float(v.abs().max()) for v in (dg, du)) < 2 ** 16        # two parts of 8 bits hold them, and half's range
    for mag in parts.sums(dg.abs(), du.abs(), X.abs(), Wg.abs(), Wu.abs()):
        assert float(mag.max()) < 2 ** 24                               # FP32 holds every partial sum


@pytest.mark.parametrize("t", parts.BITS, ids=str)
@pytest.mark.parametrize("case", parts.CASES, ids=str)
def test_two_parts_give_the_exact_gradients(case, t):
    args = parts.inputs(case)
    for a, b in zip(parts.planted(*args, t, ""), parts.sums(*parts.kept(*args), *args[1:])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("how", parts.PLANTS)
@pytest.mark.parametrize("t", parts.BITS, ids=str)
@pytest.mark.parametrize("case", parts.CASES, ids=str)
def test_a_mistake_shows(case, t, how):
    args = parts.inputs(case)
    want = parts.sums(*parts.kept(*args), *args[1:])
    wrong = parts.planted(*args, t, how)
    # (a mistake in one of the two parts leaves the other's weight gradient right)
    for i, name in enumerate(("dX", "dWg", "dWu")):
        if (how, name) in (("drop dG's", "dWu"), ("drop dU's", "dWg")):
            continue
        assert (wrong[i].to(t) != want[i].to(t)).any(), name
