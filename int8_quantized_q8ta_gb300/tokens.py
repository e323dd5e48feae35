"""Rows with a scale for each token (the last part of include/q8ta.h):
activations quantized as they come, the int8 products and the gated pair of
projections on them, and the gradients through int8 weights.

Argument marshalling only, like the rest of the package; imported by it.  The
products take float rows, which they quantize, or int8 rows with their scales.
Float rows that require a gradient get it where the transposed weight is given:
the call is then recorded for autograd, and keeps the int8 rows and their
scales (linear_gated) or its output under relu (linear_per_token), never the
float rows.
"""
from __future__ import annotations

import dataclasses
import functools
from typing import Optional, Tuple

import torch

from . import Q8_ERR_SHAPE, Q8Error, _check, _lib, _need, _stream
from .rows import (_DTYPE, PackedTileWeight, _arg, _dtype_code, _out, _shape, _space, _vector_arg)

_HALVES = (torch.float16, torch.bfloat16)


def _float_code(dtype, name: str) -> int:
    code = _DTYPE.get(dtype)
    if code is None or code == 3:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return code


def _half_arg(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(dtype code, address) of a float16 or bfloat16 matrix."""
    code = _dtype_code(t, name)
    if code not in (1, 2):
        raise TypeError(f"{name} must be float16 or bfloat16, got {t.dtype}")
    at = _arg(t, t.dtype, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {tuple(t.shape)}")
    return code, at


def quantize_per_token(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Float rows [M, K] to int8, each with its own scale (see
    q8_quantize_per_token): returns (q int8 [M, K], scales float32 [M])."""
    code = _float_code(getattr(x, "dtype", type(x)), "x")
    at = _arg(x, x.dtype, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be [M, K], got {tuple(x.shape)}")
    M, K = x.shape
    q = _out(out, (M, K), torch.int8, x.device)
    scales = _out(scales, (M,), torch.float32, x.device, "scales")
    _check(_lib.q8_quantize_per_token(at, code, M, K, q.data_ptr(), scales.data_ptr(), _stream(x)),
           "q8_quantize_per_token")
    return q, scales


def dequantize_per_token(q: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 rows [M, K] times their scales, in a float type."""
    at = _arg(q, torch.int8, "q")
    if q.dim() != 2:
        raise ValueError(f"q must be [M, K], got {tuple(q.shape)}")
    M, K = q.shape
    s = _arg(scales, torch.float32, "scales")
    _shape(scales, (M,), "scales")
    code = _float_code(out_dtype, "out_dtype")
    out = _out(out, (M, K), out_dtype, q.device)
    _check(_lib.q8_dequantize_per_token(at, s, M, K, code, out.data_ptr(), _stream(q)),
           "q8_dequantize_per_token")
    return out


# What is recorded for autograd: the result, already computed, as a function of
# the float rows.

class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, packed_t, weight_scales, relu):
        ctx.packed_t, ctx.x_dtype = packed_t, x.dtype
        ctx.save_for_backward(weight_scales, *((y,) if relu else ()))
        ctx.mark_dirty(y)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        weight_scales, *y = ctx.saved_tensors
        dx = linear_per_token_backward(dy.contiguous(), ctx.packed_t, weight_scales,
                                       y=y[0] if y else None)
        return dx.to(ctx.x_dtype), None, None, None, None


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h, x_q, x_scales, packed, packed_t, weight_scales, bias, activation):
        ctx.packed, ctx.packed_t, ctx.activation, ctx.x_dtype = packed, packed_t, activation, x.dtype
        ctx.save_for_backward(x_q, x_scales, weight_scales, *(() if bias is None else (bias,)))
        ctx.mark_dirty(h)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x_q, x_scales, weight_scales, *bias = ctx.saved_tensors
        dx = linear_gated_backward(dh.contiguous(), x_q, x_scales, ctx.packed, ctx.packed_t,
                                   weight_scales, bias[0] if bias else None,
                                   activation=ctx.activation)
        return (dx.to(ctx.x_dtype),) + (None,) * 8


def _recorded(x, weight_scales, bias, packed_t, out_dtype) -> bool:
    """Whether this call is recorded; what cannot be differentiated is refused."""
    if not torch.is_grad_enabled():
        return False
    for t, name in ((weight_scales, "weight_scales"), (bias, "bias")):
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} gets no gradient here: pass it detached")
    if not x.requires_grad:
        return False
    if packed_t is None:
        raise ValueError("x requires a gradient: give packed_t, or pass x detached")
    if out_dtype not in _HALVES:
        raise TypeError("gradients are float16 or bfloat16: x requires one and out_dtype is "
                        f"{out_dtype}")
    return True


def _rows(x, x_scales, K: int) -> Tuple[int, int, int, int]:
    """(dtype code, address, M, address of the scales) of either form of rows."""
    code = _dtype_code(x, "x")
    at = _arg(x, x.dtype, "x")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M, {K}], got {tuple(x.shape)}")
    M = x.shape[0]
    if code == 3:
        if x_scales is None:
            raise ValueError("int8 x comes with x_scales")
        s = _arg(x_scales, torch.float32, "x_scales")
        _shape(x_scales, (M,), "x_scales")
        return code, at, M, s
    if x_scales is not None:
        raise ValueError("float x is quantized here: x_scales must be None")
    return code, at, M, 0


def _out_dtype(x, out_dtype):
    if out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype is torch.int8 else x.dtype
    return out_dtype, _float_code(out_dtype, "out_dtype")


# (sizes depend on the device's SMs)
@functools.lru_cache(maxsize=4096)
def _bytes(query: str, a: int, b: int, c: int, device: int) -> int:
    with torch.cuda.device(device):
        return getattr(_lib, query)(a, b, c)


def linear_per_token(x, x_scales, packed: PackedTileWeight, weight_scales, bias, activation="none",
                     out_dtype=None, packed_t: Optional[PackedTileWeight] = None, out=None,
                     workspace=None):
    """int8 x [M, K] with x_scales [M], or float x (quantized here, x_scales
    None), times an int8 weight [N, K], scales for each token and channel (see
    q8_linear_per_token): weight_scales and bias float32 [N]; out [M, N] of
    out_dtype (by default x's own, bfloat16 for int8 x).  packed_t
    (pack_tile_weight of the transposed weight) records the call for autograd
    where x requires a gradient."""
    N, K = packed.N, packed.K
    if packed.E != 1:
        raise ValueError(f"the packed weight has {packed.E} groups, this product takes one")
    code, at, M, s = _rows(x, x_scales, K)
    _need(weight_scales, torch.float32, "weight_scales")
    scales = _vector_arg(weight_scales, (N,), "weight_scales")
    b = _vector_arg(bias, (N,), "bias")
    out_dtype, out_code = _out_dtype(x, out_dtype)
    record = _recorded(x, weight_scales, bias, packed_t, out_dtype)
    if packed_t is not None and (packed_t.E, packed_t.N, packed_t.K) != (1, K, N):
        raise ValueError(f"packed_t must be of a {K}x{N} weight")
    out = _out(out, (M, N), out_dtype, x.device)
    nbytes = _bytes("q8_linear_per_token_workspace_bytes", M, K, N, x.get_device())
    ws = _space(nbytes, x.device, workspace)
    _check(_lib.q8_linear_per_token(at, code, M, K, 0, s, packed.data.data_ptr(), N, scales, b,
                                    activation.encode(), out_code, out.data_ptr(), ws.data_ptr(),
                                    nbytes, _stream(x)), "q8_linear_per_token")
    if record:
        out = _Linear.apply(x, out, packed_t, weight_scales, activation == "relu")
    return out


def linear_per_token_backward(dy, packed_t: PackedTileWeight, weight_scales, y=None, out=None,
                              workspace=None):
    """The gradient of linear_per_token's rows (see
    q8_linear_per_token_backward): dy [M, N] float16 or bfloat16, y the forward
    output under relu; out [M, K] of dy's type."""
    code, at = _half_arg(dy, "dy")
    K, N = packed_t.N, packed_t.K
    if packed_t.E != 1:
        raise ValueError(f"the packed weight has {packed_t.E} groups, this product takes one")
    M = dy.shape[0]
    _shape(dy, (M, N), "dy")
    y_at = 0
    if y is not None:
        y_at = _arg(y, dy.dtype, "y")
        _shape(y, (M, N), "y")
    _need(weight_scales, torch.float32, "weight_scales")
    scales = _vector_arg(weight_scales, (N,), "weight_scales")
    out = _out(out, (M, K), dy.dtype, dy.device)
    nbytes = _bytes("q8_linear_per_token_backward_workspace_bytes", M, N, K, dy.get_device())
    ws = _space(nbytes, dy.device, workspace)
    _check(_lib.q8_linear_per_token_backward(at, code, M, N, y_at, packed_t.data.data_ptr(), K,
                                             scales, out.data_ptr(), ws.data_ptr(), nbytes,
                                             _stream(dy)), "q8_linear_per_token_backward")
    return out


# ---------------------------------------------------------------------------
# the gated pair
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class PackedGatedWeight:
    """A gated pair's int8 weights [N, K] in tiles (see q8_gated_pack_weight):
    ``data`` is a uint8 CUDA buffer, ``transposed`` the gradient's layout."""
    data: torch.Tensor
    N: int
    K: int
    transposed: bool


def _pack_gated(gate, up, transposed: bool) -> PackedGatedWeight:
    _need(gate, torch.int8, "gate")
    _need(up, torch.int8, "up")
    if gate.dim() != 2:
        raise ValueError(f"gate must be [N, K], got {tuple(gate.shape)}")
    _shape(up, gate.shape, "up")
    N, K = gate.shape
    nbytes = _lib.q8_gated_packed_weight_bytes(N, K, int(transposed))
    if nbytes == 0:
        raise Q8Error(Q8_ERR_SHAPE, "q8_gated_packed_weight_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=gate.device)
    _check(_lib.q8_gated_pack_weight(gate.data_ptr(), up.data_ptr(), N, K, int(transposed),
                                     buf.data_ptr(), nbytes, _stream(gate)), "q8_gated_pack_weight")
    return PackedGatedWeight(buf, N, K, transposed)


def pack_gated_weight(gate: torch.Tensor, up: torch.Tensor) -> PackedGatedWeight:
    """Pack a gated pair's int8 weights [N, K] once, for linear_gated."""
    return _pack_gated(gate, up, False)


def pack_gated_weight_t(gate: torch.Tensor, up: torch.Tensor) -> PackedGatedWeight:
    """The same weights once more, transposed, for their gradient."""
    return _pack_gated(gate, up, True)


def _gated_args(packed, packed_t, weight_scales, bias) -> Tuple[int, int, int, int]:
    """(N, K) of the pair and the addresses of its scales and biases."""
    if packed.transposed:
        raise ValueError("packed is a transposed weight (pack_gated_weight_t)")
    N, K = packed.N, packed.K
    if packed_t is not None and (not packed_t.transposed or (packed_t.N, packed_t.K) != (N, K)):
        raise ValueError(f"packed_t must come from pack_gated_weight_t of {N}x{K} weights")
    _need(weight_scales, torch.float32, "weight_scales")
    return (N, K, _vector_arg(weight_scales, (2, N), "weight_scales"),
            _vector_arg(bias, (2, N), "bias"))


def linear_gated(x, x_scales, packed: PackedGatedWeight, weight_scales, bias, activation="silu",
                 out_dtype=None, packed_t: Optional[PackedGatedWeight] = None, out=None,
                 workspace=None):
    """act(gate projection) * up projection of int8 x [M, K] with x_scales [M],
    or of float x (quantized here, x_scales None), in one product (see
    q8_linear_gated): weight_scales float32 [2, N], bias float32 [2, N] or None,
    the gate's first; activation "silu", "gelu" or "relu"; out [M, N] of
    out_dtype (by default x's own, bfloat16 for int8 x).  packed_t
    (pack_gated_weight_t) records the call for autograd where x requires a
    gradient; it then keeps the int8 rows and their scales."""
    N, K, scales, b = _gated_args(packed, packed_t, weight_scales, bias)
    code, at, M, s = _rows(x, x_scales, K)
    out_dtype, out_code = _out_dtype(x, out_dtype)
    record = _recorded(x, weight_scales, bias, packed_t, out_dtype)
    out = _out(out, (M, N), out_dtype, x.device)
    nbytes = _bytes("q8_linear_gated_workspace_bytes", M, K, N, x.get_device())
    ws = _space(nbytes, x.device, workspace)
    q_at = 0
    if record:
        x_q = torch.empty((M, K), dtype=torch.int8, device=x.device)
        x_scales = torch.empty(M, dtype=torch.float32, device=x.device)
        q_at, s = x_q.data_ptr(), x_scales.data_ptr()
    _check(_lib.q8_linear_gated(at, code, M, K, q_at, s, packed.data.data_ptr(), N, scales, b,
                                activation.encode(), out_code, out.data_ptr(), ws.data_ptr(), nbytes,
                                _stream(x)), "q8_linear_gated")
    if record:
        out = _Gated.apply(x, out, x_q, x_scales, packed, packed_t, weight_scales, bias, activation)
    return out


def linear_gated_backward(dh, x, x_scales, packed: PackedGatedWeight, packed_t: PackedGatedWeight,
                          weight_scales, bias, activation="silu", out=None, workspace=None):
    """The gradient of linear_gated's rows from the int8 rows x [M, K] and their
    scales (see q8_linear_gated_backward): dh [M, N] float16 or bfloat16; out
    [M, K] of dh's type."""
    code, at = _half_arg(dh, "dh")
    if packed_t is None:
        raise ValueError("the gradient needs packed_t (pack_gated_weight_t)")
    N, K, scales, b = _gated_args(packed, packed_t, weight_scales, bias)
    M = dh.shape[0]
    _shape(dh, (M, N), "dh")
    q = _arg(x, torch.int8, "x")
    _shape(x, (M, K), "x")
    s = _arg(x_scales, torch.float32, "x_scales")
    _shape(x_scales, (M,), "x_scales")
    out = _out(out, (M, K), dh.dtype, dh.device)
    nbytes = _bytes("q8_linear_gated_backward_workspace_bytes", M, K, N, dh.get_device())
    ws = _space(nbytes, dh.device, workspace)
    _check(_lib.q8_linear_gated_backward(at, code, M, N, q, s, K, packed.data.data_ptr(),
                                         packed_t.data.data_ptr(), scales, b, activation.encode(),
                                         out.data_ptr(), ws.data_ptr(), nbytes, _stream(dh)),
           "q8_linear_gated_backward")
    return out
