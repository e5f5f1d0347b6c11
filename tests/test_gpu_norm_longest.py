"""The norm's backward pass in rows of 2^28 numbers and more: the sums of dW's parts
need more blocks of 64 columns than one grid of their workgroups may have. Sums
are of whole numbers, and compared for equality."""
import pytest

torch = pytest.importorskip("torch")
import fp32_gemm_tuning_amd as sg  # noqa: E402

pytestmark = pytest.mark.gpu
K = (1 << 28) + 70


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    d = torch.device("cuda:0")
    if torch.cuda.mem_get_info(d)[0] < 32 << 30:
        pytest.skip("less than 32 GiB of memory free")
    return d


def test_gradients_of_the_longest_rows(dev):
    print("[gpu] longest rows", flush=True)
    t = torch.bfloat16
    at = torch.arange(K, device=dev, dtype=torch.int32)
    # 1 to 5 by turns of 64, signs by turns: every 16 bytes of a row sum to zero, and so does dY N
    v = ((1 + (at >> 6) % 5) * (1 - 2 * (at & 1))).to(t)
    del at
    H, W = torch.ones(2, K, dtype=t, device=dev), torch.ones(K, dtype=t, device=dev)
    dY = torch.stack((v, -2 * v))
    rstd = torch.tensor([0.5, 2.0], device=dev)
    dX, dW = sg.rms_norm_backward(dY, H, W, rstd)
    assert torch.equal(dW, v * -3.5)                                   # 0.5 v + 2 (-2 v)
    assert torch.equal(dX[0], v * 0.5) and torch.equal(dX[1], v * -4)
    del dX, dW
    none, dW = sg.rms_norm_backward(dY, H, W, rstd, dX=False)
    assert none is None and torch.equal(dW, v * -3.5)
    dW.fill_(7)
    sg.rms_norm_backward(dY[:0], H[:0], W, rstd[:0], dX=False, dW=dW)
    assert (dW == 0).all()
    del H, W, dY, dW, v
    torch.cuda.empty_cache()
