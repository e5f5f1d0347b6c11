"""Timed cases of the feed-forward operators: the gated block (glu), its
backward pass, and products with 4-bit weights (w4).

listed() gives the cases, draw() more of the same ranges, prepare() a case's
inputs, run() one pass, work() the bytes and operations it cannot do without,
exact() its result in 64 bits. With `own` false run() computes the plain form
in elementary torch operations; with `own` true it calls the package.

The operators (X: M x K activations, weights row-major with one row of K
inputs for each output feature):
  glu         H = act(X Wg^T) * (X Wu^T)
  glu_train   the same and, for a given dH, dX, dWg and dWu
  w4          Y = X W^T with W in 4 bits, W[n][k] = (q - zero) * scale, one
              scale (and zero point) for each group of `group` inputs of a row
  w4_glu      glu with both weights in 4 bits
  w4_pack     a weight matrix to 4 bits and back: scales, zero points, values
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
SMOOTH = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one token through a small layer: the smallest call, latency counts
        {"name": "glu token f32", "op": "glu", "dtype": "f32", "act": "silu", "M": 1, "F": 256, "K": 256},
        # a decoding batch of sixteen sequences: every weight read once for few rows
        {"name": "glu rows bf16", "op": "glu", "dtype": "bf16", "act": "silu", "M": 16, "F": 8192, "K": 4096},
        # a prompt: both projections are large products
        {"name": "glu prompt bf16", "op": "glu", "dtype": "bf16", "act": "silu", "M": 4096, "F": 8192, "K": 4096},
        # a training step at sizes no tile divides, in single precision
        {"name": "glu_train ragged f32", "op": "glu_train", "dtype": "f32", "act": "gelu", "M": 1000, "F": 1531, "K": 777},
        # a training step of a large layer: the largest case
        {"name": "glu_train large bf16", "op": "glu_train", "dtype": "bf16", "act": "silu", "M": 4096, "F": 8192, "K": 4096},
        # a short sequence through an odd layer in half precision
        {"name": "glu_train short f16", "op": "glu_train", "dtype": "f16", "act": "gelu_tanh", "M": 77, "F": 1000, "K": 511},
        # decoding one sequence: the weights' bytes are the work
        {"name": "w4 token bf16", "op": "w4", "dtype": "bf16", "M": 1, "F": 8192, "K": 8192, "group": 128, "zeros": False},
        # the near-GEMV shape of this repository, sixteen rows in single precision, with zero points
        {"name": "w4 rows f32", "op": "w4", "dtype": "f32", "M": 16, "F": 8192, "K": 8192, "group": 64, "zeros": True},
        # decoding one sequence through the gated block
        {"name": "w4_glu token bf16", "op": "w4_glu", "dtype": "bf16", "act": "silu", "M": 1, "F": 8192, "K": 4096, "group": 128, "zeros": False},
        # a batch of drafts through odd sizes, small groups, zero points
        {"name": "w4_glu rows f16", "op": "w4_glu", "dtype": "f16", "act": "gelu_tanh", "M": 33, "F": 4091, "K": 4092, "group": 32, "zeros": True},
        # preparing a large layer's weights
        {"name": "w4_pack f32", "op": "w4_pack", "dtype": "f32", "F": 8192, "K": 8192, "group": 128, "zeros": False},
        # a small odd layer, with zero points and groups that end past the row
        {"name": "w4_pack ragged bf16", "op": "w4_pack", "dtype": "bf16", "F": 1531, "K": 777, "group": 64, "zeros": True},
    ]


def _log_size(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("glu", "glu_train", "w4", "w4_glu", "w4_pack"))
    case = {"op": op, "dtype": rng.choice(("f32", "bf16", "f16"))}
    if op in ("glu", "w4_glu"):
        case["act"] = rng.choice(SMOOTH + ("relu",))
    elif op == "glu_train":
        case["act"] = rng.choice(SMOOTH)   # relu's derivative jumps at 0: no two summation orders agree there
    case["F"], case["K"] = _log_size(rng, 64, 8192), _log_size(rng, 64, 8192)
    if op in ("glu", "glu_train"):
        most = 4096 * 4096 * 8192 // (case["F"] * case["K"])
        case["M"] = _log_size(rng, 1, min(4096, most))
    elif op != "w4_pack":
        case["M"] = _log_size(rng, 1, 256)
    if op.startswith("w4"):
        case["group"], case["zeros"] = rng.choice((32, 64, 128, 256)), rng.random() < 0.5
    return case


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _groups(W, group):
    """W's rows cut into groups (the last one filled with zeros), as 64-bit."""
    n, k = W.shape
    g = -(-k // group)
    out = torch.zeros(n, g * group, dtype=torch.float64, device=W.device)
    out[:, :k] = W
    return out.view(n, g, group)


def _quantise(W, group, zeros, dtype):
    """(bytes, scales, zero points or None): the definition of the 4-bit
    form, in 64 bits around the scale as stored (a quotient next to a half
    must not be rounded twice)."""
    n, k = W.shape
    w = _groups(W, group)
    if zeros:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).to(dtype)
    else:
        lo = None
        s = (w.abs().amax(-1) / 7).to(dtype)
    d = s.double()
    d = torch.where(d == 0, torch.ones_like(d), d)
    z = (-lo / d).round().clamp(0, 15) if zeros else torch.full_like(d, 8.0)
    q = ((w / d[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).view(n, -1)[:, :k]
    if k % 2:
        q = torch.nn.functional.pad(q, (0, 1))
    return q[:, 0::2] | (q[:, 1::2] << 4), s, z.to(dtype) if zeros else None


def _normal(shape, gen, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, F, K = DTYPES[case["dtype"]], case["F"], case["K"]
    state = dict(case)
    if case["op"] == "w4_pack":
        state["W"] = _normal((F, K), gen, t, K ** -0.5)
        return state
    state["X"] = _normal((case["M"], K), gen, t)
    if case["op"] in ("glu", "glu_train"):
        state["Wg"] = _normal((F, K), gen, t, K ** -0.5)
        state["Wu"] = _normal((F, K), gen, t, K ** -0.5)
        if case["op"] == "glu_train":
            state["dH"] = _normal((case["M"], F), gen, t)
    else:
        for name in ("a", "b") if case["op"] == "w4_glu" else ("a",):
            W = _normal((F, K), gen, torch.float32, K ** -0.5)
            state[name] = _quantise(W, case["group"], case["zeros"], t)
    state["out"] = torch.empty(case["M"], F, dtype=t, device="cuda")
    return state


# --------------------------------------------------------------------------
# The plain form: 32 bits, rounded once at the end
# --------------------------------------------------------------------------
def _act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    if kind == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 0.7071067811865476))
    if kind == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))
    return torch.clamp(g, min=0.0)


def _act_slope(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(g * 0.7071067811865476)) + g * 0.3989422804014327 * torch.exp(-0.5 * g * g)
    if kind == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 0.134145 * g * g)
    return (g > 0).to(g.dtype)


def _unpack(packed, k, group):
    """The 4-bit weights' values in 32 bits."""
    b, s, z = packed
    q = torch.stack((b & 15, b >> 4), dim=-1).view(b.shape[0], -1)[:, :k].float()
    s = s.float().repeat_interleave(group, dim=1)[:, :k]
    z = 8.0 if z is None else z.float().repeat_interleave(group, dim=1)[:, :k]
    return (q - z) * s


def _plain(st):
    op, t = st["op"], DTYPES[st["dtype"]]
    if op == "w4_pack":
        p = _quantise(st["W"], st["group"], st["zeros"], t)
        values = _unpack(p, st["K"], st["group"]).to(t)
        return {"W": values, "scales": p[1]} | ({"zeros": p[2]} if st["zeros"] else {})
    x = st["X"].float()
    if op == "w4":
        return (x @ _unpack(st["a"], st["K"], st["group"]).T).to(t)
    if op == "w4_glu":
        g = x @ _unpack(st["a"], st["K"], st["group"]).T
        u = x @ _unpack(st["b"], st["K"], st["group"]).T
        return (_act(g, st["act"]) * u).to(t)
    wg, wu = st["Wg"].float(), st["Wu"].float()
    g, u = x @ wg.T, x @ wu.T
    a = _act(g, st["act"])
    h = (a * u).to(t)
    if op == "glu":
        return h
    dh = st["dH"].float()
    dg, du = dh * u * _act_slope(g, st["act"]), dh * a
    return {"H": h, "dX": (dg @ wg + du @ wu).to(t), "dWg": (dg.T @ x).to(t), "dWu": (du.T @ x).to(t)}


# --------------------------------------------------------------------------
# The package's operators
# --------------------------------------------------------------------------
def _own(st):
    import fp32_gemm_tuning_amd as sg

    op = st["op"]
    if op == "glu":
        return sg.glu(st["X"], st["Wg"], st["Wu"], st["act"], out=st["out"])
    if op == "glu_train":
        pre = torch.empty(st["M"], 2 * st["F"], dtype=torch.float32, device="cuda")
        h = sg.glu(st["X"], st["Wg"], st["Wu"], st["act"], out=st["out"], preact=pre)
        dx, dwg, dwu = sg.glu_backward(st["dH"], st["X"], st["Wg"], st["Wu"], pre, st["act"])
        return {"H": h, "dX": dx, "dWg": dwg, "dWu": dwu}
    if op == "w4_pack":
        p = sg.w4_quantize(st["W"], st["group"], zeros=st["zeros"])
        return {"W": sg.w4_dequantize(p), "scales": p.scales} | ({"zeros": p.zeros} if st["zeros"] else {})
    a = sg.W4(*st["a"], st["K"], st["group"])
    if op == "w4":
        return sg.w4_matmul(st["X"], a, out=st["out"])
    return sg.w4_glu(st["X"], a, sg.W4(*st["b"], st["K"], st["group"]), st["act"], out=st["out"])


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# What a pass cannot do without: inputs read once, outputs written once
# --------------------------------------------------------------------------
def work(case):
    e, F, K = BYTES[case["dtype"]], case["F"], case["K"]
    packed = 0
    if case["op"].startswith("w4"):
        packed = F * ((K + 1) // 2) + F * -(-K // case["group"]) * e * (2 if case["zeros"] else 1)
    if case["op"] == "w4_pack":
        # one pass over W for the packed form; the values come from that
        return {"bytes": 2 * F * K * e + 2 * packed, "flops": 4 * F * K}
    M = case["M"]
    if case["op"] == "w4":
        return {"bytes": packed + e * (M * K + M * F), "flops": 2 * M * F * K}
    if case["op"] == "w4_glu":
        return {"bytes": 2 * packed + e * (M * K + M * F), "flops": 4 * M * F * K}
    if case["op"] == "glu":
        return {"bytes": e * (M * K + 2 * F * K + M * F), "flops": 4 * M * F * K}
    return {"bytes": e * (2 * M * K + 4 * F * K + 2 * M * F), "flops": 12 * M * F * K}


# --------------------------------------------------------------------------
# The definition in 64 bits, apart from the plain form
# --------------------------------------------------------------------------
def _gate64(g, kind):
    """(act(g), act'(g)) in 64 bits."""
    if kind == "silu":
        e = torch.exp(-g.abs())
        s = torch.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * s, s + g * s * (1 - s)
    if kind == "gelu":
        cdf = torch.special.erfc(-g / math.sqrt(2)) / 2
        return g * cdf, cdf + g * torch.exp(-g ** 2 / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = torch.special.expit(2 * c * (g + 0.044715 * g ** 3))   # (1 + tanh(v)) / 2
        return g * s, s + 2 * c * g * s * (1 - s) * (1 + 3 * 0.044715 * g ** 2)
    return torch.where(g > 0, g, 0.0), torch.where(g > 0, 1.0, 0.0).double()


def _weights64(packed, k, group):
    b, s, z = packed
    n = b.shape[0]
    w = torch.empty(n, 2 * b.shape[1], dtype=torch.float64, device=b.device)
    w[:, 0::2], w[:, 1::2] = b % 16, b // 16
    at = torch.arange(k, device=b.device) // group
    return (w[:, :k] - (8 if z is None else z.double()[:, at])) * s.double()[:, at]


def exact(case, seed):
    st = prepare(case, seed)
    op, k = st["op"], st["K"]
    if op == "w4_pack":
        W, t = st["W"].double(), DTYPES[st["dtype"]]
        at = torch.arange(k, device=W.device) // st["group"]
        index = at.expand(W.shape)
        top = torch.zeros(W.shape[0], int(at[-1]) + 1, dtype=torch.float64, device=W.device)
        hi = top.scatter_reduce(1, index, W, "amax")
        lo = top.scatter_reduce(1, index, W, "amin")
        scale = (hi - lo) / 15 if st["zeros"] else torch.maximum(hi, -lo) / 7
        kept = scale.to(t).double()     # the scale as it is kept is part of the definition
        s = kept[:, at]
        if st["zeros"]:
            z = torch.where(kept > 0, torch.round(-lo / kept), 0.0).clamp(0, 15)
            level = torch.where(s > 0, torch.round(W / s), 0.0)
            level = torch.minimum(torch.maximum(level, -z[:, at]), 15 - z[:, at])
            return {"W": level * s, "scales": scale, "zeros": z}
        level = torch.where(s > 0, torch.round(W / s), 0.0).clamp(-8, 7)
        return {"W": level * s, "scales": scale}
    x = st["X"].double()
    if op == "w4":
        return torch.mm(x, _weights64(st["a"], k, st["group"]).t())
    if op == "w4_glu":
        g = torch.mm(x, _weights64(st["a"], k, st["group"]).t())
        return _gate64(g, st["act"])[0] * torch.mm(x, _weights64(st["b"], k, st["group"]).t())
    wg, wu = st["Wg"].double(), st["Wu"].double()
    g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    a, slope = _gate64(g, st["act"])
    if op == "glu":
        return a * u
    du = st["dH"].double()
    dg = du * u * slope
    du = du * a
    return {"H": a * u, "dX": torch.mm(dg, wg).add_(torch.mm(du, wu)),
            "dWg": torch.mm(dg.t(), x), "dWu": torch.mm(du.t(), x)}
