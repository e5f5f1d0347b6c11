"""Inputs of the gated block's backward pass whose dG and dU need two parts of a
16-bit type and whose sums are exact in FP32 in any order, the exact gradients,
and the same with mistakes in the second parts (on the CPU, in 64 bits)."""
import torch

# M, F, K, largest |X|, |W| and |dH|. M * F <= 16384 (dG and dU in two parts);
# dX and the weights' gradients split over their slices or not; rows of whole
# 16-byte chunks or not, and shorter than one.
CASES = [(9, 130, 77, 5, 5, 90), (128, 128, 40, 5, 5, 90), (16, 64, 96, 5, 5, 60), (40, 33, 50, 5, 5, 100),
         (30, 100, 5, 9, 9, 99), (300, 50, 64, 5, 5, 60), (1, 700, 87, 20, 2, 90), (250, 65, 33, 4, 5, 90)]
BITS = {torch.bfloat16: 8, torch.float16: 11}
PLANTS = ("drop", "negate", "exchange", "drop dG's", "drop dU's")


def inputs(case):
    """(dH, X, Wg, Wu), whole numbers in 64 bits, for relu."""
    M, F, K, x, w, h = case
    gen = torch.Generator().manual_seed(1000 * M + F)
    draw = lambda shape, top: torch.randint(-top, top + 1, shape, generator=gen).double()   # noqa: E731
    return draw((M, F), h), draw((M, K), x), draw((F, K), w), draw((F, K), w)


def kept(dH, X, Wg, Wu):
    """dG and dU."""
    g, u = X @ Wg.T, X @ Wu.T
    return dH * u * (g > 0), dH * g.clamp(min=0)


def sums(dg, du, X, Wg, Wu):
    return dg @ Wg + du @ Wu, dg.T @ X, du.T @ X


def planted(dH, X, Wg, Wu, t, how):
    """The gradients with a mistake in how the second parts of dG and dU are used."""
    dg, du = kept(dH, X, Wg, Wu)
    g1, u1 = dg.to(t).double(), du.to(t).double()
    g2, u2 = (dg - g1).to(t).double(), (du - u1).to(t).double()
    if how == "drop":
        g2, u2 = 0 * g2, 0 * u2
    elif how == "negate":
        g2, u2 = -g2, -u2
    elif how == "exchange":
        g2, u2 = u2, g2
    elif how == "drop dG's":
        g2 = 0 * g2
    elif how == "drop dU's":
        u2 = 0 * u2
    return sums(g1 + g2, u1 + u2, X, Wg, Wu)
