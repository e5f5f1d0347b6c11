"""Timed cases of the norm that precedes a feed-forward block and of that
block's 8-bit form: root-mean-square norm with the residual's addition
(rms_norm), its backward pass, its 8-bit output (rms_norm_i8), matrices in 8
bits (i8_quantize), their product (i8_matmul) and the gated block over them
(i8_glu).

listed() gives the cases, draw() more of the same ranges, prepare() a case's
inputs, run() one pass, work() the bytes and operations it cannot do without,
exact() its result in 64 bits. With `own` false run() computes the plain form
in elementary torch operations; with `own` true it calls the package.

The operators (X: M x K, a weight has one row of K inputs for each output
feature, S holds one FP32 scale for each row of a matrix in 8 bits):
  norm        H = X + R (rounded to the type; R may be absent: H = X),
              Y = H rstd W with rstd = 1 / sqrt(mean(H^2) + eps), row by row
  norm_train  the same and, for given dY and the gradient D that reaches H
              from behind, N = H rstd,
              dX = D + rstd (dY W - N mean(dY W N)), dW = sum over rows of dY N
  norm_i8     H, and Y in 8 bits: q = round(127 H W / max|H W|),
              S = max|H W| rstd / 127; the values are q S
  i8_pack     a matrix to 8 bits and back: q = round(127 X / max|X|), S = max|X| / 127
  i8          Y = Sx Sw (sum of qx qw)
  i8_glu      act(X Wg^T) * (X Wu^T) of matrices in 8 bits
Halves round to even. Values in 8 bits are returned as the values they stand for.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
NORMS = ("norm", "norm_train", "norm_i8")
EPS = 1e-6


def listed():
    return [
        # one token between two blocks while decoding: the smallest call, latency counts
        {"name": "norm token bf16", "op": "norm", "dtype": "bf16", "M": 1, "K": 4096, "residual": True},
        # the heads of a prompt's queries, each normed by itself: short rows, many of them
        {"name": "norm heads f16", "op": "norm", "dtype": "f16", "M": 131072, "K": 128, "residual": False},
        # a training step over a large batch of tokens
        {"name": "norm_train large bf16", "op": "norm_train", "dtype": "bf16", "M": 4096, "K": 8192, "residual": True},
        # a training step at sizes no tile divides, in single precision
        {"name": "norm_train ragged f32", "op": "norm_train", "dtype": "f32", "M": 1000, "K": 1531, "residual": False},
        # a decoding batch of sixteen sequences on its way into a product in 8 bits
        {"name": "norm_i8 rows bf16", "op": "norm_i8", "dtype": "bf16", "M": 16, "K": 8192, "residual": True},
        # a prompt on the same way, kept in single precision, of an odd length
        {"name": "norm_i8 prompt f32", "op": "norm_i8", "dtype": "f32", "M": 2047, "K": 4096, "residual": True},
        # preparing a large layer's weights
        {"name": "i8_pack f32", "op": "i8_pack", "dtype": "f32", "M": 8192, "K": 8192},
        # a block's activations before its second product, odd sizes
        {"name": "i8_pack ragged bf16", "op": "i8_pack", "dtype": "bf16", "M": 1531, "K": 777},
        # decoding one sequence: the weights' bytes are the work
        {"name": "i8 token bf16", "op": "i8", "dtype": "bf16", "M": 1, "F": 8192, "K": 8192},
        # a short prompt at sizes no tile divides
        {"name": "i8 ragged f32", "op": "i8", "dtype": "f32", "M": 1000, "F": 1531, "K": 777},
        # a batch of drafts through the gated block, odd sizes
        {"name": "i8_glu rows f16", "op": "i8_glu", "dtype": "f16", "act": "gelu_tanh", "M": 33, "F": 4091, "K": 4092},
        # a prompt through the gated block: the largest case
        {"name": "i8_glu prompt bf16", "op": "i8_glu", "dtype": "bf16", "act": "silu", "M": 4096, "F": 8192, "K": 4096},
    ]


def _log_size(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(NORMS + ("i8_pack", "i8", "i8_glu"))
    case = {"op": op, "dtype": rng.choice(("f32", "bf16", "f16"))}
    if op in NORMS or op == "i8_pack":
        case["K"] = _log_size(rng, 64, 16384)
        case["M"] = _log_size(rng, 1, 4096 * 8192 * 2 // (BYTES[case["dtype"]] * case["K"]))
        if op in NORMS:
            case["residual"] = rng.random() < 0.5
        return case
    if op == "i8_glu":
        case["act"] = rng.choice(("silu", "gelu", "gelu_tanh", "relu"))
    case["F"], case["K"] = _log_size(rng, 64, 8192), _log_size(rng, 64, 8192)
    most = 4096 * 4096 * 8192 // (case["F"] * case["K"])
    case["M"] = _log_size(rng, 1, min(4096, most))
    return case


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _normal(shape, gen, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _stream(shape, gen, dtype):
    """Rows of a residual stream: a few channels are far larger than the rest."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * 2.0
    big = torch.rand(shape[1], generator=gen, device="cuda") < 0.004
    return (x * torch.where(big, 20.0, 1.0)).to(dtype)


def _pack(v):
    """(q, scales) of a matrix: the definition of the 8-bit form in 64 bits (a
    quotient next to a half must not be rounded twice)."""
    v = v.double()
    top = v.abs().amax(1)
    d = torch.where(top > 0, top, torch.ones_like(top))
    return (v * 127.0 / d[:, None]).round().to(torch.int8), (top / 127.0).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, M, K = DTYPES[case["dtype"]], case["M"], case["K"]
    state = dict(case)
    if case["op"] == "i8_pack":
        state["X"] = _normal((M, K), gen, t)
    elif case["op"] in NORMS:
        state["X"] = _stream((M, K), gen, t)
        state["R"] = _stream((M, K), gen, t) if case["residual"] else None
        state["W"] = (1.0 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(t)
        if case["op"] == "norm_train":
            state["dY"] = _normal((M, K), gen, t)
            state["D"] = _normal((M, K), gen, t) if case["residual"] else None
        if case["op"] != "norm_i8":
            state["out"] = torch.empty(M, K, dtype=t, device="cuda")
        state["total"] = torch.empty(M, K, dtype=t, device="cuda") if case["residual"] else None
    else:
        state["x"] = _pack(_normal((M, K), gen, t))
        for name in ("a", "b") if case["op"] == "i8_glu" else ("a",):
            state[name] = _pack(_normal((case["F"], K), gen, torch.float32, K ** -0.5))
        state["out"] = torch.empty(M, case["F"], dtype=t, device="cuda")
    return state


# --------------------------------------------------------------------------
# The plain form: 32 bits (64 for quotients that are rounded to whole
# numbers), rounded once at the end
# --------------------------------------------------------------------------
def _act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    if kind == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * 0.7071067811865476))
    if kind == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))
    return torch.clamp(g, min=0.0)


def _values(q, scales, dtype):
    return (q.float() * scales[:, None]).to(dtype)


def _product(x, w):
    """Whole numbers of at most 127: every partial sum below 2^24 is exact."""
    return (x[0].float() @ w[0].float().T) * x[1][:, None] * w[1]


def _plain(st):
    op, t = st["op"], DTYPES[st["dtype"]]
    if op == "i8_pack":
        q, s = _pack(st["X"])
        return {"X": _values(q, s, t), "scales": s}
    if op == "i8":
        return _product(st["x"], st["a"]).to(t)
    if op == "i8_glu":
        return (_act(_product(st["x"], st["a"]), st["act"]) * _product(st["x"], st["b"])).to(t)
    total = st["X"] if st["R"] is None else (st["X"].float() + st["R"].float()).to(t)
    h, w = total.float(), st["W"].float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    sums = {} if st["R"] is None else {"H": total}
    if op == "norm_i8":
        v = total.double() * st["W"].double()
        q, _ = _pack(v)
        s = (v.abs().amax(1) * rstd[:, 0].double() / 127.0).float()
        return {"Y": _values(q, s, t), "scales": s} | sums
    n = h * rstd
    y = (n * w).to(t)
    if op == "norm":
        return {"Y": y} | sums
    dy = st["dY"].float()
    g = dy * w
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if st["D"] is not None:
        dx = dx + st["D"].float()
    return {"Y": y, "dX": dx.to(t), "dW": (dy * n).sum(0).to(t)} | sums


# --------------------------------------------------------------------------
# The package's operators
# --------------------------------------------------------------------------
def _own(st):
    import fp32_gemm_tuning_amd as sg

    op, t = st["op"], DTYPES[st["dtype"]]
    if op == "i8_pack":
        p = sg.i8_quantize(st["X"])
        return {"X": sg.i8_dequantize(p, t), "scales": p.scales}
    if op == "i8":
        return sg.i8_matmul(sg.I8(*st["x"]), sg.I8(*st["a"]), out=st["out"])
    if op == "i8_glu":
        return sg.i8_glu(sg.I8(*st["x"]), sg.I8(*st["a"]), sg.I8(*st["b"]), st["act"], out=st["out"])
    sums = {} if st["R"] is None else {"H": st["total"]}
    if op == "norm_i8":
        p = sg.rms_norm_i8(st["X"], st["W"], EPS, residual=st["R"], total=st["total"])
        return {"Y": sg.i8_dequantize(p, t), "scales": p.scales} | sums
    if op == "norm":
        return {"Y": sg.rms_norm(st["X"], st["W"], EPS, residual=st["R"], out=st["out"], total=st["total"])} | sums
    rstd = torch.empty(st["M"], dtype=torch.float32, device="cuda")
    y = sg.rms_norm(st["X"], st["W"], EPS, residual=st["R"], out=st["out"], total=st["total"], rstd=rstd)
    h = st["X"] if st["R"] is None else st["total"]
    dx, dw = sg.rms_norm_backward(st["dY"], h, st["W"], rstd, dH=st["D"])
    return {"Y": y, "dX": dx, "dW": dw} | sums


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# What a pass cannot do without: inputs read once, outputs written once
# --------------------------------------------------------------------------
def work(case):
    e, M, K, op = BYTES[case["dtype"]], case["M"], case["K"], case["op"]
    if op == "i8_pack":
        # into 8 bits, and from there to the values
        return {"bytes": 2 * M * K * e + 2 * M * K + 8 * M, "flops": 3 * M * K}
    if op in ("i8", "i8_glu"):
        F, n = case["F"], 2 if op == "i8_glu" else 1
        return {"bytes": M * K + 4 * M + n * (F * K + 4 * F) + e * M * F, "flops": 2 * n * M * F * K}
    ways = 2 if case["residual"] else 0          # R read, H written
    if op == "norm":
        return {"bytes": e * ((2 + ways) * M * K + K), "flops": 4 * M * K}
    if op == "norm_i8":
        # q is written, and read again for the values
        return {"bytes": e * ((2 + ways) * M * K + K) + 2 * M * K + 8 * M, "flops": 6 * M * K}
    # the forward pass, then H, dY (and D) read, dX and dW written
    back = 3 + (1 if case["residual"] else 0)
    return {"bytes": e * ((2 + ways + back) * M * K + 3 * K) + 8 * M, "flops": 14 * M * K}


# --------------------------------------------------------------------------
# The definition in 64 bits, apart from the plain form
# --------------------------------------------------------------------------
def _gate64(g, kind):
    if kind == "silu":
        return g * torch.special.expit(g)
    if kind == "gelu":
        return g * torch.special.erfc(-g / math.sqrt(2)) / 2
    if kind == "gelu_tanh":
        return g * torch.special.expit(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    return torch.where(g > 0, g, 0.0)


def _levels64(v):
    """Each row's whole numbers and its largest magnitude."""
    top, _ = v.abs().max(dim=1, keepdim=True)
    return torch.where(top > 0, torch.round(127 * v / top), 0.0), top


def _matrix64(p):
    return p[0].double() * p[1].double().view(-1, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op, t = st["op"], DTYPES[st["dtype"]]
    if op == "i8_pack":
        n, top = _levels64(st["X"].double())
        return {"X": n * (top / 127), "scales": (top / 127).squeeze(1)}
    if op in ("i8", "i8_glu"):
        x = _matrix64(st["x"])
        g = torch.mm(x, _matrix64(st["a"]).t())
        return g if op == "i8" else _gate64(g, st["act"]) * torch.mm(x, _matrix64(st["b"]).t())
    h = st["X"].double()
    out = {}
    if st["R"] is not None:
        out["H"] = h + st["R"].double()
        h = out["H"].to(t).double()      # the sum as it is kept is part of the definition
    K = h.shape[1]
    r = 1 / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / K + EPS)
    w = st["W"].double().view(1, -1)
    if op == "norm_i8":
        n, top = _levels64(h * w)
        s = top * r / 127
        return {"Y": n * s, "scales": s.squeeze(1)} | out
    u = h * r
    out["Y"] = u * w
    if op == "norm":
        return out
    dy = st["dY"].double()
    along = torch.linalg.vecdot(dy * w, u).view(-1, 1) / K
    out["dX"] = r * (dy * w) - r * u * along
    if st["D"] is not None:
        out["dX"] = out["dX"] + st["D"].double()
    out["dW"] = torch.mv((dy * u).t(), torch.ones(h.shape[0], dtype=torch.float64, device=h.device))
    return out
