"""64-bit references and error bounds for the tests of the norm and of matrices
in 8 bits (plain torch on float64; nothing of the library's)."""
import torch

from ffn_ref import HALF_STEP, TINY, act, act_eval_error, sum_error

ONE = 2.0 ** -24   # one FP32 rounding, relative


def total(X, R):
    """H: the FP32 sum, rounded to the type (X itself where R is None)."""
    return X if R is None else (X.float() + R.float()).to(X.dtype)


def rstd(H, eps):
    h = H.double()
    return 1 / torch.sqrt((h * h).sum(1) / max(H.shape[1], 1) + eps)


def rstd_error(K):
    """Relative: half of the sum's (the root), a division, an addition and a
    reciprocal root of one step each."""
    return sum_error(K) / 2 + 4 * ONE


def norm(H, W, eps):
    return H.double() * rstd(H, eps)[:, None] * W.double()


def norm_bound(H, W, eps, dtype):
    """|Y - exact|: rstd's error, two products in FP32, one rounding to the type (and
    FP32's smallest number, times W, where the first product loses bits there)."""
    y = norm(H, W, eps).abs()
    b = y * (rstd_error(H.shape[1]) + 2.1 * ONE) + TINY["f32"] * (1 + W.double().abs())
    return b + HALF_STEP[dtype] * (y + b) + TINY[dtype]


def levels(V):
    """(q, max) of rows in 64 bits; rows with an infinity or NaN are zeros with a NaN."""
    v = V.double()
    top = v.abs().amax(1) if v.shape[1] else v.new_zeros(v.shape[0])
    bad = ~torch.isfinite(v).all(1)
    d = torch.where((top > 0) & ~bad, top, 1.0)
    q = torch.where(((top > 0) & ~bad)[:, None], torch.round(127 * v / d[:, None]), 0.0)
    return q.to(torch.int8), torch.where(bad, float("nan"), top)


def near_half(V, width):
    """Where 127 v / max lies within `width` of a half."""
    v = V.double()
    x = 127 * v / v.abs().amax(1, keepdim=True)
    return ((x - torch.floor(x)) - 0.5).abs() < width


def norm_grads(dY, H, W, r, dH=None):
    """(dX, dW) for given rstd `r`, in 64 bits."""
    dy, h, w, r = dY.double(), H.double(), W.double(), r.double()[:, None]
    n, g = h * r, dy * w
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    return dx if dH is None else dx + dH.double(), (dy * n).sum(0)


def norm_grads_bounds(dY, H, W, r, dH, dtype):
    """N and dY W are one rounding each; the row's mean is a sum of K products of
    those, divided; dX takes a multiply-add, a product and an addition more. dW sums M
    products."""
    dy, h, w, r = dY.double().abs(), H.double().abs(), W.double().abs(), r.double()[:, None].abs()
    M, K = H.shape
    n, g = h * r, dy * w
    c = (g * n).mean(1, keepdim=True)
    ec = c * (sum_error(K) + 4 * ONE)
    full = r * (g + n * c)
    d = dH.double().abs() if dH is not None else 0.0
    bx = r * n * ec + 6 * ONE * (full + d) + 4 * TINY["f32"] * (1 + r + n + w)
    bx = bx + HALF_STEP[dtype] * (full + d + bx) + TINY[dtype]
    mag = (dy * n).sum(0)
    bw = mag * (sum_error(M) + 2 * ONE) + M * TINY["f32"]
    return bx, bw + HALF_STEP[dtype] * (mag + bw) + TINY[dtype]


def product(x, w):
    """Sx Sw sum(qx qw) of (q, scales) pairs, in 64 bits (sums exact)."""
    return (x[0].double() @ w[0].double().T) * x[1].double()[:, None] * w[1].double()


PRODUCT_ERROR = 3.1 * ONE    # the sum and two scales, a rounding each


def product_bound(y, dtype):
    b = y.abs() * PRODUCT_ERROR + TINY["f32"]
    return b + HALF_STEP[dtype] * (y.abs() + b) + TINY[dtype]


def glu(x, wg, wu, kind):
    return act(product(x, wg), kind)[0] * product(x, wu)


# The hardware's exponential of 16-bit gates: 2^-21 + |x| 2^-23 relative.
def glu_bound(x, wg, wu, kind, dtype):
    g, u = product(x, wg), product(x, wu)
    a = act(g, kind)[0]
    eg, eu = g.abs() * PRODUCT_ERROR + TINY["f32"], u.abs() * PRODUCT_ERROR + TINY["f32"]
    ev = act_eval_error(g, kind) + (2.0 ** -20 if dtype != "f32" else 0.0)
    b = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + (a * u).abs() * (ev + 2.0 ** -23)
    return b + HALF_STEP[dtype] * ((a * u).abs() + b) + TINY[dtype]
