"""64-bit references, error bounds and operand layouts for the feed-forward
tests (plain torch on float64; nothing of the library's)."""
import math

import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # one rounding, relative
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}     # smallest subnormal
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def act(g, kind):
    """(act, act') in 64 bits."""
    if kind == "silu":
        s = torch.special.expit(g)
        return g * s, s + g * s * (1 - s)
    if kind == "gelu":
        c = torch.special.erfc(-g / math.sqrt(2)) / 2
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = torch.special.expit(2 * c * (g + 0.044715 * g ** 3))
        return g * s, s + g * s * (1 - s) * 2 * c * (1 + 0.134145 * g * g)
    return g.clamp(min=0), (g > 0).double()


def act_eval_error(g, kind):
    """Relative error of act and of each term of act' as computed in FP32: a few
    roundings (2^-24 each; library exp, erfc within 2 steps), and the rounded
    argument of the exponential or erfc, whose relative error the function
    magnifies by its logarithmic derivative: |g| for exp(-g), up to
    2 x^2 + 2 = g^2 + 2 for erfc and exp(-g^2/2), 2|v| for exp(-2v)."""
    a = g.abs()
    grow = {"silu": a, "gelu": a * a + 2, "gelu_tanh": 2 * (0.8 * (a + 0.045 * a ** 3)) * 4, "relu": 0 * a}[kind]
    return (12 + 2 * grow) * 2.0 ** -24


def glu(X, Wg, Wu, kind):
    g, u = X @ Wg.T, X @ Wu.T
    return act(g, kind)[0] * u


def sum_error(n):
    """Relative to the sum of magnitudes: n products summed in FP32 in any
    order, each addition off by at most one step (2^-23) even where it
    truncates."""
    return (n + 2) * 2.0 ** -23


def glu_bound(X, Wg, Wu, kind, dtype):
    """Elementwise bound of |H - exact|. Slopes of the activations are at
    most 1.13 in magnitude."""
    g, u = X @ Wg.T, X @ Wu.T
    e = sum_error(X.shape[1])
    eg, eu = e * (X.abs() @ Wg.abs().T), e * (X.abs() @ Wu.abs().T)
    a = act(g, kind)[0]
    b = 1.13 * eg * (u.abs() + eu) + a.abs() * eu + (a * u).abs() * (act_eval_error(g, kind) + 2.0 ** -23)
    return b + HALF_STEP[dtype] * ((a * u).abs() + b) + TINY[dtype]


def glu_grads(dH, X, Wg, Wu, kind):
    g, u = X @ Wg.T, X @ Wu.T
    a, s = act(g, kind)
    dg, du = dH * u * s, dH * a
    return dg @ Wg + du @ Wu, dg.T @ X, du.T @ X


def glu_grads_bounds(dH, X, Wg, Wu, kind, dtype):
    """Elementwise bounds for dX, dWg and dWu (smooth activations: second
    derivatives are at most 1 in magnitude). dG and dU are rounded once to the
    type, then summed in FP32, and the sums rounded once. Up to 16384 values dG
    and dU are kept in two parts, the second a rounding of what the first left:
    their error is half a step of half a step."""
    r, t = HALF_STEP[dtype], TINY[dtype]
    rd = r * r if dtype != "f32" and dH.numel() <= 16384 else r
    g, u = X @ Wg.T, X @ Wu.T
    e = sum_error(X.shape[1])
    eg, eu = e * (X.abs() @ Wg.abs().T), e * (X.abs() @ Wu.abs().T)
    a, s = act(g, kind)
    h, ev = dH.abs(), act_eval_error(g, kind)
    # act' is a sum of two terms: the errors of both count with their sizes,
    # at most 1 and |g| * 0.5 each (the second's factor falls off with |g|).
    size = s.abs() + 1.2
    edg = h * ((u.abs() + eu) * (eg + size * (ev + 2.0 ** -22)) + s.abs() * eu)
    edu = h * (1.13 * eg + a.abs() * (ev + 2.0 ** -23))
    dg, du = dH * u * s, dH * a
    edg = edg + rd * (dg.abs() + edg) + t
    edu = edu + rd * (du.abs() + edu) + t
    M, F = dH.shape

    def close(err, mag, n):
        b = err + sum_error(n) * (mag + err)
        return b + r * (mag + b) + t

    bx = close(edg @ Wg.abs() + edu @ Wu.abs(), dg.abs() @ Wg.abs() + du.abs() @ Wu.abs(), 2 * F)
    bg = close(edg.T @ X.abs(), dg.abs().T @ X.abs(), M)
    bu = close(edu.T @ X.abs(), du.abs().T @ X.abs(), M)
    return bx, bg, bu


def w4_values(q, scales, zeros, K, group):
    """The matrix that 4-bit weights stand for, in 64 bits."""
    n = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)[:, :K].double()
    at = torch.arange(K, device=q.device) // group
    z = 8.0 if zeros is None else zeros.double()[:, at]
    return (n - z) * scales.double()[:, at]


def w4_bound(X, q, scales, zeros, K, group, dtype):
    """Elementwise bound of |Y - exact| for Y = X W^T. The kernels sum q x (or
    (16 + q) x) and z x (or (16 + z) x) apart and subtract, so the magnitudes
    that roundings act on are (q + 16 + |z + 16|) |x| s."""
    n = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)[:, :K].double()
    at = torch.arange(K, device=q.device) // group
    z = torch.full_like(n, 8.0) if zeros is None else zeros.double()[:, at]
    s = scales.double()[:, at]
    mag = X.abs() @ ((n + 16 + (z + 16).abs()) * s.abs()).T
    b = sum_error(K + 16) * mag
    return b, b + HALF_STEP[dtype] * ((X @ ((n - z) * s).T).abs() + b) + TINY[dtype]


def quantise(W, group, zeros, dtype):
    """(q, scales, zeros) by the definition, in 64 bits, one group at a time."""
    F, K = W.shape
    G = -(-K // group)
    q = torch.zeros(F, (K + 1) // 2, dtype=torch.uint8, device=W.device)
    n = torch.zeros(F, K + K % 2, dtype=torch.float64, device=W.device)
    S = torch.empty(F, G, dtype=dtype, device=W.device)
    Z = torch.empty(F, G, dtype=dtype, device=W.device) if zeros else None
    for g in range(G):
        w = W[:, g * group:(g + 1) * group].double()
        lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
        s = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7)
        s = torch.where(torch.isfinite(w).all(1), s, float("nan")).to(dtype)
        S[:, g] = s
        s = s.double()
        ok = s > 0
        z = torch.where(ok, torch.round(-lo / s), 0.0).clamp(0, 15) if zeros else torch.full_like(s, 8.0)
        if zeros:
            Z[:, g] = z.to(dtype)
        v = torch.where(ok[:, None], torch.round(w / s[:, None]), 0.0) + z[:, None]
        n[:, g * group:g * group + w.shape[1]] = v.clamp(0, 15)
    n = n.to(torch.uint8)
    q.copy_(n[:, 0::2] | (n[:, 1::2] << 4))
    return q, S, Z


def laid_out(x, pad=0, offset=0, fill=float("nan")):
    """`x` as a view of a buffer of its own with `pad` elements behind each
    row and `offset` before the first, all of them `fill`."""
    rows, cols = x.shape
    flat = torch.full((offset + rows * (cols + pad) + 64,), fill, dtype=x.dtype, device=x.device)
    v = flat.as_strided((rows, cols), (cols + pad, 1), offset)
    v.copy_(x)
    return v, flat


def around_untouched(flat, view, fill_is_nan=True):
    """Whether everything of `flat` outside `view` still holds the fill."""
    left = flat.clone()
    left.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(float("nan"))
    return bool(torch.isnan(left).all())
