"""The 64-bit references of the norm and of the 8-bit form against hand-worked
numbers and automatic differentiation, without a GPU."""
import pytest

torch = pytest.importorskip("torch")
import i8_ref  # noqa: E402


def test_levels_by_hand():
    # largest 254: quotients are v / 2, halves go to the even neighbour
    v = torch.tensor([[254.0, 1, 3, 5, -1, -3, 253, -254], [0, 0, 0, 0, 0, 0, 0, 0],
                      [1, float("inf"), 0, 0, 0, 0, 0, 0], [1, float("nan"), 0, 0, 0, 0, 0, 0]])
    q, top = i8_ref.levels(v)
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, 126, -127] and top[0] == 254
    assert (q[1:] == 0).all() and top[1] == 0 and top[2:].isnan().all()
    assert i8_ref.near_half(v[:1], 1e-9)[0].tolist() == [False, True, True, True, True, True, True, False]


def test_product_by_hand():
    x = (torch.tensor([[1, -2, 127]], dtype=torch.int8), torch.tensor([0.5]))
    w = (torch.tensor([[3, 4, -128], [0, 1, 0]], dtype=torch.int8), torch.tensor([2.0, -4.0]))
    assert i8_ref.product(x, w).tolist() == [[3 - 8 - 127 * 128.0, 4.0]]


@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_gradients_against_autograd(with_dh):
    g = torch.Generator().manual_seed(3)
    H, dY, D = (torch.randn(5, 17, generator=g, dtype=torch.float64) for _ in range(3))
    W = torch.randn(17, generator=g, dtype=torch.float64)
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-3) * w
    assert torch.allclose(y.detach(), i8_ref.norm(H, W, 1e-3), rtol=1e-14)
    ((dY * y).sum() + ((D * h).sum() if with_dh else 0)).backward()
    dx, dw = i8_ref.norm_grads(dY, H, W, i8_ref.rstd(H, 1e-3), D if with_dh else None)
    assert torch.allclose(dx, h.grad, rtol=1e-12, atol=1e-13) and torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("mistake", [
    lambda dy, h, w, r: (r * (dy * w - h * (dy * w * h * r).mean(1, keepdim=True)), None),      # N taken as H
    lambda dy, h, w, r: (r * (dy * w - h * r * (dy * w * h * r).sum(1, keepdim=True)), None),   # a sum for the mean
    lambda dy, h, w, r: (r * (dy * w), None),                                                     # no projection
    lambda dy, h, w, r: (None, (dy * h).sum(0)),                                                  # rstd left out
    lambda dy, h, w, r: (None, (dy * h * r * w).sum(0))],                                         # W not taken off
    ids=["H for N", "sum for mean", "no projection", "no rstd", "with W"])
def test_bounds_tell_a_wrong_gradient(mistake):
    # Inputs of the GPU tests' kind: a wrong formula leaves the bounds.
    g = torch.Generator().manual_seed(4)
    H, dY = (torch.randn(9, 300, generator=g, dtype=torch.float64) * 3 for _ in range(2))
    W = 1 + 0.3 * torch.randn(300, generator=g, dtype=torch.float64)
    r = i8_ref.rstd(H, 1e-5)
    right = i8_ref.norm_grads(dY, H, W, r)
    for dtype in ("f32", "bf16", "f16"):
        bounds = i8_ref.norm_grads_bounds(dY, H, W, r, None, dtype)
        for wrong, good, b in zip(mistake(dY, H, W, r[:, None]), right, bounds):
            if wrong is not None:
                assert ((wrong - good).abs() > b).float().mean() > 0.1
