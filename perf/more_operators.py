"""The operators of an int8 feed-forward block whose activations carry a scale
for each token, as cases to measure: rows quantized and back, products with
scales for each token and channel, the gated pair of projections, and the
gradients through both.

Each case runs in two forms on the same inputs: a plain one of elementary
torch operations in 32 bits, and (``own``) this package's entry points.

kinds of case
  rows         float rows to int8 with each row's own scale, and back
  linear       rows times an int8 weight, scales for each token and channel;
               float rows are quantized on the way, int8 ones come with scales
  linear_grad  the gradient of the rows behind such a product
  gated        act(rows x gate) * (rows x up) with int8 weights
  gated_grad   its gradient, from the rows as int8 with their scales
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rows(name, M, K, dtype):
    return {"name": name, "kind": "rows", "M": M, "K": K, "dtype": dtype}


def _linear(name, M, N, K, x, out, bias=True, relu=False):
    return {"name": name, "kind": "linear", "M": M, "N": N, "K": K, "x": x, "out": out, "bias": bias, "relu": relu}


def _linear_grad(name, M, N, K, dtype, relu=False):
    return {"name": name, "kind": "linear_grad", "M": M, "N": N, "K": K, "dtype": dtype, "relu": relu}


def _gated(name, M, N, K, x, out, act="silu", bias=False):
    return {"name": name, "kind": "gated", "M": M, "N": N, "K": K, "x": x, "out": out, "act": act, "bias": bias}


def _gated_grad(name, M, N, K, dtype, act="silu", bias=False):
    return {"name": name, "kind": "gated_grad", "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias}


def listed():
    return [
        # one token of a decode step
        _rows("rows_1x4096_bf16", 1, 4096, "bf16"),
        # a training batch's hidden rows, kept in 8 bits until their backward pass
        _rows("rows_8192x11008_bf16", 8192, 11008, "bf16"),
        # the projection back to the model's width for one token
        _linear("linear_1_4096x11008_bf16", 1, 4096, 11008, "bf16", "bf16", bias=False),
        # a decode batch whose rows were quantized before, outputs in full precision
        _linear("linear_24_11008x4096_i8_f32", 24, 11008, 4096, "i8", "f32"),
        # a prompt
        _linear("linear_2048_4096x11008_bf16", 2048, 4096, 11008, "bf16", "bf16"),
        # odd sizes, half precision, rows cut off by the activation
        _linear_grad("linear_grad_777_1003x1234_f16", 777, 1003, 1234, "f16", relu=True),
        # a training batch
        _linear_grad("linear_grad_2048_4096x11008_bf16", 2048, 4096, 11008, "bf16"),
        # both projections and the gate for one token
        _gated("gated_1_11008x4096_bf16", 1, 11008, 4096, "bf16", "bf16"),
        # a decode batch of odd sizes, another gate, biases
        _gated("gated_33_2749x1031_f16", 33, 2749, 1031, "f16", "f16", act="gelu", bias=True),
        # a prompt
        _gated("gated_2048_11008x4096_bf16", 2048, 11008, 4096, "bf16", "bf16"),
        # a short batch of a narrow block
        _gated_grad("gated_grad_200_1376x1000_f16", 200, 1376, 1000, "f16", act="gelu", bias=True),
        # a training batch
        _gated_grad("gated_grad_1024_11008x4096_bf16", 1024, 11008, 4096, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if c["M"] * c["K"] <= 8192 * 11008 and work(c)["flops"] <= 3.6e11:
            return c


def _draw(rng):
    kind = rng.choice(["rows", "linear", "linear", "linear_grad", "gated", "gated", "gated_grad"])
    if kind == "rows":
        c = _rows("", _log(rng, 1, 16384), _log(rng, 64, 16384), rng.choice(["f32", "bf16", "f16"]))
        del c["name"]
        return c
    M, N, K = _log(rng, 1, 4096), _log(rng, 64, 11008), _log(rng, 64, 11008)
    x, out, half = rng.choice(["i8", "f32", "bf16", "f16"]), rng.choice(["f32", "bf16", "f16"]), rng.choice(["bf16", "f16"])
    act, bias, relu = rng.choice(["silu", "silu", "gelu", "relu"]), rng.random() < 0.5, rng.random() < 0.3
    if kind == "linear":
        c = _linear("", M, N, K, x, out, bias=bias, relu=relu)
    elif kind == "linear_grad":
        c = _linear_grad("", M, N, K, half, relu=relu)
    elif kind == "gated":
        c = _gated("", M, N, K, x, out, act=act, bias=bias)
    else:
        c = _gated_grad("", M, N, K, half, act=act, bias=bias)
    del c["name"]
    return c


def work(case):
    c = case
    M, K = c["M"], c["K"]
    if c["kind"] == "rows":  # the way back comes later: it reads the int8 rows again
        return {"bytes": 2 * M * K * (BYTES[c["dtype"]] + 1) + 8 * M, "flops": 0}
    N, per_channel = c["N"], 8 if c.get("bias") else 4
    if c["kind"] == "linear_grad":
        b = BYTES[c["dtype"]]
        return {"bytes": M * N * b * (2 if c["relu"] else 1) + N * K + 4 * N + M * K * b, "flops": 2 * M * N * K}
    if c["kind"] == "gated_grad":  # both projections once more, and their transposed products
        b = BYTES[c["dtype"]]
        return {"bytes": M * K + 4 * M + M * N * b + 4 * N * K + 2 * per_channel * N + M * K * b, "flops": 8 * M * N * K}
    rows = M * K * BYTES[c["x"]] + (4 * M if c["x"] == "i8" else 0)
    n = 2 * N if c["kind"] == "gated" else N
    return {"bytes": rows + n * (K + per_channel) + M * N * BYTES[c["out"]], "flops": 2 * M * n * K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, shape, scale=1.0):
    return scale * torch.randn(shape, generator=g, device=g.device)


def _activations(g, M, K):
    """Rows of a normalised layer: tokens of different size, a few channels far above the others."""
    x = _normal(g, (M, K)) * (0.5 + torch.rand((M, 1), generator=g, device=g.device))
    return x * torch.where(torch.rand(K, generator=g, device=g.device) < 0.01, 6.0, 1.0)


def _quantized(g, M, K):
    """Such rows as int8 with their scales, as a program has them from an earlier layer."""
    x = _activations(g, M, K)
    s = x.abs().amax(1) / torch.full((), 127.0, device=x.device)
    return torch.round(x / s[:, None]).clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    M, K = c["M"], c["K"]
    if c["kind"] == "rows":
        s["x"] = _activations(g, M, K).to(DTYPES[c["dtype"]])
        return s
    N, grad, gated = c["N"], c["kind"].endswith("_grad"), c["kind"].startswith("gated")
    each = 2 if gated else 1
    s["w"] = torch.randint(-127, 128, (each, N, K), generator=g, device=g.device, dtype=torch.int8)
    # outputs of about unit size: int8 weights spread by some 73
    s["ws"] = (0.5 + torch.rand((each, N), generator=g, device=g.device)) / (73.0 * math.sqrt(K))
    s["b"] = _normal(g, (each, N), 0.3) if c.get("bias") else None
    if not gated:
        s["ws"], s["b"] = s["ws"][0], s["b"][0] if c.get("bias") else None
    if c["kind"] != "linear_grad":
        x = "i8" if grad else c["x"]
        s["x"], s["xs"] = _quantized(g, M, K) if x == "i8" else (_activations(g, M, K).to(DTYPES[x]), None)
    if grad:
        s["dy"] = _normal(g, (M, N), 0.05).to(DTYPES[c["dtype"]])
        if c.get("relu"):
            s["y"] = _normal(g, (M, N)).clamp(min=0).to(DTYPES[c["dtype"]])
    if own:  # weights are laid out once, when a program loads them
        import int8_quantized_q8ta_gb300 as q8
        if gated:
            s["packed"] = q8.pack_gated_weight(s["w"][0], s["w"][1])
            if grad:
                s["packed_t"] = q8.pack_gated_weight_t(s["w"][0], s["w"][1])
        elif grad:
            s["packed_t"] = q8.pack_tile_weight(s["w"][0].t().contiguous())
        else:
            s["packed"] = q8.pack_tile_weight(s["w"][0])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_OWN if own else _PLAIN)[state["c"]["kind"]](state, state["c"])


def _own_rows(s, c):
    import int8_quantized_q8ta_gb300 as q8
    q, scales = q8.quantize_per_token(s["x"])
    return {"values": q8.dequantize_per_token(q, scales, out_dtype=s["x"].dtype), "scales": scales}


def _own_linear(s, c):
    import int8_quantized_q8ta_gb300 as q8
    return q8.linear_per_token(s["x"], s["xs"], s["packed"], s["ws"], s["b"],
                               activation="relu" if c["relu"] else "none", out_dtype=DTYPES[c["out"]])


def _own_linear_grad(s, c):
    import int8_quantized_q8ta_gb300 as q8
    return q8.linear_per_token_backward(s["dy"], s["packed_t"], s["ws"], y=s["y"] if c["relu"] else None)


def _own_gated(s, c):
    import int8_quantized_q8ta_gb300 as q8
    return q8.linear_gated(s["x"], s["xs"], s["packed"], s["ws"], s["b"], activation=c["act"],
                           out_dtype=DTYPES[c["out"]])


def _own_gated_grad(s, c):
    import int8_quantized_q8ta_gb300 as q8
    return q8.linear_gated_backward(s["dy"], s["x"], s["xs"], s["packed"], s["packed_t"], s["ws"], s["b"],
                                    activation=c["act"])


_OWN = {"rows": _own_rows, "linear": _own_linear, "linear_grad": _own_linear_grad, "gated": _own_gated,
        "gated_grad": _own_gated_grad}


def _plain_quantize(x):
    """(integers in 32-bit floats, scales): the scale, its reciprocal and the product each rounded once."""
    x = x.float()
    scale = x.abs().amax(1) / torch.full((), 127.0, device=x.device)  # (a number would be multiplied by its reciprocal)
    inv = (1.0 / scale.double()).float()
    return torch.round(x * inv[:, None]).clamp(-127, 127), scale


def _plain_x(s):
    return (s["x"].float(), s["xs"]) if s["xs"] is not None else _plain_quantize(s["x"])


def _plain_product(q, scale, w, ws, b):
    v = (q @ w.float().t()) * scale[:, None] * ws
    return v if b is None else v + b


def _plain_act(g, act):
    """The activation and its derivative."""
    if act == "relu":
        return g.clamp(min=0), (g > 0).float()
    if act == "silu":
        sigma = 1 / (1 + torch.exp(-g))
        return g * sigma, sigma * (1 + g * (1 - sigma))
    phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _plain_rows(s, c):
    q, scale = _plain_quantize(s["x"])
    return {"values": (q * scale[:, None]).to(s["x"].dtype), "scales": scale}


def _plain_linear(s, c):
    v = _plain_product(*_plain_x(s), s["w"][0], s["ws"], s["b"])
    return (v.clamp(min=0) if c["relu"] else v).to(DTYPES[c["out"]])


def _plain_linear_grad(s, c):
    dy = s["dy"].float()
    if c["relu"]:
        dy = torch.where(s["y"] > 0, dy, torch.zeros((), device=dy.device))
    return ((dy * s["ws"]) @ s["w"][0].float()).to(s["dy"].dtype)


def _plain_pair(s):
    q, scale = _plain_x(s)
    return [_plain_product(q, scale, s["w"][i], s["ws"][i], None if s["b"] is None else s["b"][i]) for i in (0, 1)]


def _plain_gated(s, c):
    g, u = _plain_pair(s)
    return (_plain_act(g, c["act"])[0] * u).to(DTYPES[c["out"]])


def _plain_gated_grad(s, c):
    g, u = _plain_pair(s)
    a, da = _plain_act(g, c["act"])
    dh = s["dy"].float()
    dx = (dh * u * da * s["ws"][0]) @ s["w"][0].float() + (dh * a * s["ws"][1]) @ s["w"][1].float()
    return dx.to(s["dy"].dtype)


_PLAIN = {"rows": _plain_rows, "linear": _plain_linear, "linear_grad": _plain_linear_grad, "gated": _plain_gated,
          "gated_grad": _plain_gated_grad}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _f32(v):
    return v.to(torch.float32).to(torch.float64)


def _quantize64(x):
    """The quantizer is defined with its roundings to 32 bits, so the integers are exact."""
    v = x.to(torch.float64)
    top = torch.maximum(v.max(dim=1).values, -v.min(dim=1).values)
    scale = _f32(top / 127)
    inv = _f32(scale.reciprocal())
    return torch.round(_f32(v * inv.unsqueeze(1))), scale


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "rows":
        q, scale = _quantize64(s["x"])
        return {"values": q * scale.unsqueeze(1), "scales": scale}
    w = s["w"].to(torch.float64)
    if c["kind"] == "linear_grad":
        dy = s["dy"].to(torch.float64)
        if c["relu"]:
            dy = dy * (s["y"] > 0)
        return torch.einsum("mn,nk->mk", dy * s["ws"].to(torch.float64), w[0])
    q, scale = (s["x"].to(torch.float64), s["xs"].to(torch.float64)) if s["xs"] is not None else _quantize64(s["x"])
    x = q * scale.unsqueeze(1)
    if c["kind"] == "linear":
        v = torch.einsum("mk,nk->mn", x, w[0]) * s["ws"].to(torch.float64)
        if s["b"] is not None:
            v = v + s["b"].to(torch.float64)
        return torch.relu(v) if c["relu"] else v
    ws = s["ws"].to(torch.float64)
    b = torch.zeros_like(ws) if s["b"] is None else s["b"].to(torch.float64)
    g = torch.einsum("mk,nk->mn", x, w[0]) * ws[0] + b[0]
    u = torch.einsum("mk,nk->mn", x, w[1]) * ws[1] + b[1]
    if c["act"] == "silu":
        t = torch.sigmoid(g)
        a, slope = g * t, t + g * t * (1 - t)
    elif c["act"] == "gelu":
        t = torch.special.ndtr(g)
        a, slope = g * t, t + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        a, slope = torch.relu(g), (g > 0).to(torch.float64)
    if c["kind"] == "gated":
        return a * u
    dh = s["dy"].to(torch.float64)
    return torch.einsum("mn,nk->mk", dh * u * slope * ws[0], w[0]) + torch.einsum("mn,nk->mk", dh * a * ws[1], w[1])
