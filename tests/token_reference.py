"""Plain forms of the operators for rows with a scale for each token, on the CPU.

Everything up to the gated pair's g and u is a fixed sequence of f32 steps on an
exact integer and is rebuilt bit for bit; what comes after is in 64 bits.
"""
import math

import torch

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def quantize(x):
    """(q int8, scales f32): a / 127, 1 / s and the product rounded once each."""
    x = x.float()
    scale = x.abs().amax(1) / torch.full((), 127.0)
    small = scale < torch.finfo(torch.float32).tiny
    scale = torch.where(small, torch.zeros(()), scale)
    inv = torch.where(small, torch.zeros((), dtype=torch.float64), 1.0 / scale.double()).float()
    return torch.round(x * inv[:, None]).to(torch.int8), scale


def product(q, xs, w, ws, b):
    """v in f32: exact accumulator, then one rounding a step."""
    acc = q.double() @ w.double().t()          # below 2^53: exact
    v = (acc.float() * xs[:, None]) * ws
    return v if b is None else v + b


def act64(g, act):
    g = g.double()
    if act == "relu":
        return g.clamp(min=0), (g > 0).double()
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    phi = torch.special.ndtr(g)
    return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def act_error(g, act):
    """(of act(g), of act'(g)): bounds on the absolute errors of the f32 forms.

    silu: exp's fast form is within 2 + 1.2 |g| units in the last place, the
    addition and the fast division within 4 more, one more product, so sigma is
    within (8 + 1.2 |g|) 2^-23 of itself; its slope is sigma + a (1 - sigma).
    gelu: erf within 2 units of at most 1, its argument within 2^-23 of itself
    (erf moves by 0.5 of that), the sum rounded: 2^-22 all told.
    """
    g = g.double().abs()
    if act == "relu":
        return torch.zeros_like(g), torch.zeros_like(g)
    if act == "silu":
        a, _ = act64(g, "silu")                # at |g|: at least as large
        rel = (8 + 1.2 * g) * 2.0 ** -23
        return (a + 1e-37) * rel, (1 + g) * rel * 2
    return g * 2.0 ** -22, (1 + g) * 2.0 ** -21


def gated(g, u, act, dtype):
    """(h in 64 bits, how far the f32 form's rounded value may be off)."""
    a, _ = act64(g, act)
    ea, _ = act_error(g, act)
    h = a * u.double()
    err = ea * u.double().abs() + h.abs() * 2.0 ** -23
    least = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}[dtype]
    return h, err * 1.01 + h.abs() * HALF_ULP[dtype] * 1.01 + least


def grad_bound(terms, extra, n, dx, dtype, floor):
    """How far a gradient may be off: `terms` sum |operand| |w| in 64 bits,
    `extra` the same of the operands' errors before they are rounded, n
    operands a sum, `floor` what the smallest operands lose.

    An operand is rounded to f16 (2^-11 of itself, or 2^-25 of its row's power
    of two, which is at most 2^-13 of the row's bound); the f32 sums of 16
    products each lose at most four units of the sum of magnitudes a step."""
    err = terms * (2.0 ** -11 + 2.0 ** -22 + (n / 16 + 8) * 2.0 ** -22) + extra + floor
    least = 2.0 ** -25 if dtype is torch.float16 else 2.0 ** -133
    return err * 1.01 + dx.abs() * HALF_ULP[dtype] * 1.01 + least


def linear_grad(dy, w, ws, y=None):
    """(dx in 64 bits, its bound)."""
    d = dy.double()
    if y is not None:
        d = torch.where(y > 0, d, torch.zeros((), dtype=torch.float64))
    t, w64 = d * ws.double(), w.double()
    dx = t @ w64
    bound = d.abs().amax(1, keepdim=True) * ws.double().abs().max()
    return dx, grad_bound(t.abs() @ w64.abs(), 0.0, w.shape[0], dx, dy.dtype,
                          2.0 ** -37 * bound * w64.abs().sum(0))


def gated_grad(dh, g, u, w, ws, act, xs, b=None):
    """(dx in 64 bits, its bound) from the f32 g and u."""
    a, slope = act64(g, act)
    ea, es = act_error(g, act)
    d, u64, w64, ws64 = dh.double(), u.double(), w.double(), ws.double()
    tg, tu = d * u64 * slope * ws64[0], d * a * ws64[1]
    dx = tg @ w64[0] + tu @ w64[1]
    terms = tg.abs() @ w64[0].abs() + tu.abs() @ w64[1].abs()
    extra = (d * u64 * es * ws64[0]).abs() @ w64[0].abs() + (d * ea * ws64[1]).abs() @ w64[1].abs()
    # (three more products in f32 before the operand's own rounding)
    extra = extra + terms * 2.0 ** -21
    # the row's bound, from the largest sum, scales and biases
    top = ws64.abs().amax(1)
    most = xs.double().abs()[:, None] * 16384 * w.shape[2]
    bias = torch.zeros(2, dtype=torch.float64) if b is None else b.double().abs().amax(1)
    bound = d.abs().amax(1, keepdim=True) * 1.25 * torch.maximum((most * top[1] + bias[1]) * top[0],
                                                                 (most * top[0] + bias[0]) * top[1])
    return dx, grad_bound(terms, extra, 2 * w.shape[1], dx, dh.dtype,
                          2.0 ** -38 * bound * w64.abs().sum((0, 1)))
