"""Rows of one batch that go through different weights (the last part of
include/q8ta.h): tokens sorted by expert and back, with weights applied, and
the gradients.

Argument marshalling only, like the rest of the package; imported by it.  Float
rows and weights that require a gradient get it: expert_gather, expert_dispatch
and expert_combine are recorded for autograd, with the gradient calls below.
The int8 products have no gradient.
"""
from __future__ import annotations

import dataclasses
import functools
from typing import Optional, Tuple

import torch

from . import Q8_ERR_SHAPE, Q8Error, _check, _lib, _need, _stream, _workspace

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}


# These calls are short on the GPU (some 5 to 20 us), so the host's part is
# kept short too: one combined check a tensor (the slow one, which names what is
# wrong, only where it fails), sizes of workspaces remembered by shape.

def _arg(t: torch.Tensor, dtype, name: str) -> int:
    """The address of a contiguous CUDA tensor of this dtype."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        _need(t, dtype, name)
    return t.data_ptr()


def _dtype_code(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16, bfloat16 or int8, got {t.dtype}")
    return code


def _shape(t: torch.Tensor, shape, name: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _out(out: Optional[torch.Tensor], shape, dtype, device, name: str = "out") -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, dtype, name)
    _shape(out, shape, name)
    return out


def _space(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is None or nbytes == 0:   # (no rows need none, whatever was given)
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return _workspace(nbytes, device, workspace)


@dataclasses.dataclass
class ExpertRoute:
    """Slots sorted by expert (see q8_expert_sort): ``order`` int32 [T*k],
    ``position`` int32 [T, k], ``offsets`` int32 [E + 1]."""
    order: torch.Tensor
    position: torch.Tensor
    offsets: torch.Tensor

    @property
    def T(self) -> int:
        return self.position.shape[0]

    @property
    def k(self) -> int:
        return self.position.shape[1]

    @property
    def E(self) -> int:
        return self.offsets.shape[0] - 1


def _route_args(route: ExpertRoute):
    """(T, k, E) and the addresses of order, position and offsets."""
    order, position, offsets = route.order, route.position, route.offsets
    o = _arg(order, torch.int32, "route.order")
    p = _arg(position, torch.int32, "route.position")
    f = _arg(offsets, torch.int32, "route.offsets")
    shape, bounds = position.shape, offsets.shape
    if len(shape) != 2 or len(bounds) != 1 or bounds[0] < 2:
        raise ValueError("route.position must be [T, k] and route.offsets [E + 1]")
    T, k = shape
    _shape(order, (T * k,), "route.order")
    return T, k, bounds[0] - 1, o, p, f


def _empty_route(expert_ids: torch.Tensor, num_experts: int) -> ExpertRoute:
    _need(expert_ids, torch.int32, "expert_ids")
    if expert_ids.dim() != 2:
        raise ValueError(f"expert_ids must be [T, k], got {tuple(expert_ids.shape)}")
    if not 1 <= num_experts <= 1024:
        raise ValueError(f"num_experts must lie in [1, 1024], got {num_experts}")
    T, k = expert_ids.shape
    return ExpertRoute(expert_ids.new_empty(T * k), torch.empty_like(expert_ids),
                       expert_ids.new_empty(num_experts + 1))


# What is recorded for autograd: the result, already computed, as a function of
# the inputs that require a gradient.

class _Gathered(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, route):
        ctx.route = route
        ctx.mark_dirty(rows)
        return rows

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_rows):
        return expert_gather_backward(d_rows.contiguous(), ctx.route), None, None


class _Combined(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, weights, y, route):
        ctx.route = route
        ctx.save_for_backward(z, weights)
        ctx.mark_dirty(y)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        dz, dw = expert_combine_backward(dy.contiguous(), *ctx.saved_tensors, ctx.route)
        return dz, dw, None, None


def expert_sort(expert_ids: torch.Tensor, num_experts: int) -> ExpertRoute:
    """Slots of int32 expert_ids [T, k] sorted by expert, stable; ids outside
    [0, num_experts) are dropped slots."""
    route = _empty_route(expert_ids, num_experts)
    T, k = expert_ids.shape
    _check(_lib.q8_expert_sort(expert_ids.data_ptr(), T, k, num_experts, route.order.data_ptr(),
                               route.position.data_ptr(), route.offsets.data_ptr(),
                               _stream(expert_ids)), "q8_expert_sort")
    return route


def expert_gather(x: torch.Tensor, route: ExpertRoute,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of x [T, H] (float32, float16, bfloat16 or int8) in sorted order,
    [T*k, H]; zeros from row offsets[E] on."""
    code = _dtype_code(x, "x")
    at = _arg(x, x.dtype, "x")
    T, k, E, _, position, offsets = _route_args(route)
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError(f"x must be [{T}, H], got {tuple(x.shape)}")
    H = x.shape[1]
    out = _out(out, (T * k, H), x.dtype, x.device)
    _check(_lib.q8_expert_gather(at, code, T, k, H, E, position, offsets, out.data_ptr(),
                                 _stream(x)), "q8_expert_gather")
    if x.requires_grad and torch.is_grad_enabled():
        out = _Gathered.apply(x, out, route)
    return out


def expert_dispatch(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int,
                    out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ExpertRoute]:
    """expert_sort, then expert_gather: returns (rows, route)."""
    code = _dtype_code(x, "x")
    at = _arg(x, x.dtype, "x")
    route = _empty_route(expert_ids, num_experts)
    T, k = expert_ids.shape
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError(f"x must be [{T}, H], got {tuple(x.shape)}")
    H = x.shape[1]
    out = _out(out, (T * k, H), x.dtype, x.device)
    _check(_lib.q8_expert_dispatch(at, code, T, H, expert_ids.data_ptr(), k, num_experts,
                                   route.order.data_ptr(), route.position.data_ptr(),
                                   route.offsets.data_ptr(), out.data_ptr(), _stream(x)),
           "q8_expert_dispatch")
    if x.requires_grad and torch.is_grad_enabled():
        out = _Gathered.apply(x, out, route)
    return out, route


def _rows_arg(t: torch.Tensor, rows: int, name: str):
    """(dtype code, address, H) of sorted rows [rows, H]."""
    code = _dtype_code(t, name)
    at = _arg(t, t.dtype, name)
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{name} must be [{rows}, H], got {tuple(t.shape)}")
    return code, at, t.shape[1]


def expert_gather_backward(d_rows: torch.Tensor, route: ExpertRoute,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gather's gradient: each token's kept rows added up in f32, [T, H]."""
    T, k, _, _, position, _ = _route_args(route)
    code, at, H = _rows_arg(d_rows, T * k, "d_rows")
    out = _out(out, (T, H), d_rows.dtype, d_rows.device)
    _check(_lib.q8_expert_gather_backward(at, code, T, k, H, position, out.data_ptr(),
                                          _stream(d_rows)), "q8_expert_gather_backward")
    return out


def expert_combine(z: torch.Tensor, weights: torch.Tensor, route: ExpertRoute,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * (slot (t, j)'s row of z), [T, H]."""
    T, k, _, _, position, _ = _route_args(route)
    code, at, H = _rows_arg(z, T * k, "z")
    w = _arg(weights, torch.float32, "weights")
    _shape(weights, (T, k), "weights")
    out = _out(out, (T, H), z.dtype, z.device)
    _check(_lib.q8_expert_combine(at, code, w, T, k, H, position, out.data_ptr(), _stream(z)),
           "q8_expert_combine")
    if (z.requires_grad or weights.requires_grad) and torch.is_grad_enabled():
        out = _Combined.apply(z, weights, out, route)
    return out


def expert_combine_backward(dy: torch.Tensor, z: torch.Tensor, weights: torch.Tensor,
                            route: ExpertRoute) -> Tuple[torch.Tensor, torch.Tensor]:
    """The combine's gradients (dz like z, dweights float32 [T, k])."""
    T, k, E, _, position, offsets = _route_args(route)
    code, at, H = _rows_arg(z, T * k, "z")
    w = _arg(weights, torch.float32, "weights")
    _shape(weights, (T, k), "weights")
    g = _arg(dy, z.dtype, "dy")
    _shape(dy, (T, H), "dy")
    dz = torch.empty((T * k, H), dtype=z.dtype, device=z.device)
    dw = torch.empty((T, k), dtype=torch.float32, device=z.device)
    _check(_lib.q8_expert_combine_backward(g, at, code, w, T, k, H, E, position, offsets,
                                           dz.data_ptr(), dw.data_ptr(), _stream(z)),
           "q8_expert_combine_backward")
    return dz, dw


# ---------------------------------------------------------------------------
# the experts' int8 products
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class PackedTileWeight:
    """int8 weights [E, N, K] in 8 KB tiles (see q8_tile_pack_weight):
    ``data`` is a uint8 CUDA buffer."""
    data: torch.Tensor
    E: int
    N: int
    K: int


def pack_tile_weight(weight: torch.Tensor) -> PackedTileWeight:
    """Pack int8 [E, N, K], or one weight [N, K], once."""
    _need(weight, torch.int8, "weight")
    if weight.dim() not in (2, 3):
        raise ValueError(f"weight must be [E, N, K] or [N, K], got {tuple(weight.shape)}")
    E, N, K = weight.shape if weight.dim() == 3 else (1, *weight.shape)
    nbytes = _lib.q8_tile_packed_weight_bytes(E, N, K)
    if nbytes == 0:
        raise Q8Error(Q8_ERR_SHAPE, "q8_tile_packed_weight_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=weight.device)
    with torch.cuda.device(weight.get_device()):
        st = _lib.q8_tile_pack_weight(weight.data_ptr(), E, N, K, buf.data_ptr(), nbytes, _stream(weight))
    _check(st, "q8_tile_pack_weight")
    return PackedTileWeight(buf, E, N, K)


# (sizes depend on the device's SMs)
@functools.lru_cache(maxsize=4096)
def _experts_space(R: int, K: int, E: int, device: int) -> int:
    with torch.cuda.device(device):
        return _lib.q8_linear_experts_workspace_bytes(R, K, E)


def _out_code(out_dtype) -> int:
    code = _DTYPE.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be float32, float16, bfloat16 or int8, got {out_dtype}")
    return code


def _vector_arg(t: Optional[torch.Tensor], shape, name: str) -> int:
    """The address of a float32 tensor of this shape, 0 for None."""
    if t is None:
        return 0
    at = _arg(t, torch.float32, name)
    _shape(t, shape, name)
    return at


def linear_experts(x, input_scale, input_zero_point, packed: PackedTileWeight, weight_scales, bias,
                   route: ExpertRoute, output_scale, output_zero_point, activation="none",
                   x_sorted=False, out_dtype=torch.int8, out=None, workspace=None):
    """Sorted rows times the int8 weight of their expert (see
    q8_linear_experts): int8 x [T, K], or [T*k, K] in sorted order with
    ``x_sorted``; weight_scales and bias float32 [E, N]; out [T*k, N]."""
    at = _arg(x, torch.int8, "x")
    T, k, E, order, _, offsets = _route_args(route)
    N, K = packed.N, packed.K
    if packed.E != E:
        raise ValueError(f"the route has {E} experts, the packed weight {packed.E}")
    _shape(x, (T * k if x_sorted else T, K), "x")
    _need(weight_scales, torch.float32, "weight_scales")
    scales = _vector_arg(weight_scales, (E, N), "weight_scales")
    b = _vector_arg(bias, (E, N), "bias")
    code = _out_code(out_dtype)
    out = _out(out, (T * k, N), out_dtype, x.device)
    nbytes = _experts_space(T * k, K, E, x.get_device())
    ws = _space(nbytes, x.device, workspace)
    _check(_lib.q8_linear_experts(
        at, int(x_sorted), T, k, K, float(input_scale), int(input_zero_point),
        packed.data.data_ptr(), E, N, scales, b, order, offsets, float(output_scale),
        int(output_zero_point), activation.encode(), code, out.data_ptr(), ws.data_ptr(), nbytes,
        _stream(x)), "q8_linear_experts")
    return out


# ---------------------------------------------------------------------------
# low-rank adapters beside a shared projection
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class PackedLora:
    """Adapters in the kernels' layout (see q8_lora_pack): ``data`` is a uint8
    CUDA buffer, ``dtype`` the type A and B came in."""
    data: torch.Tensor
    L: int
    N: int
    K: int
    r: int
    dtype: torch.dtype


def pack_lora(A: torch.Tensor, B: torch.Tensor, scaling: torch.Tensor) -> PackedLora:
    """Pack adapters A [L, r, K], B [L, N, r] (float16 or bfloat16) and
    scaling float32 [L] once.  An infinity or NaN in B makes every channel of
    its adapter's rows NaN."""
    if _dtype_code(A, "A") not in (1, 2):
        raise TypeError(f"A must be float16 or bfloat16, got {A.dtype}")
    _need(A, A.dtype, "A")
    _need(B, A.dtype, "B")
    _need(scaling, torch.float32, "scaling")
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [L, r, K] and B [L, N, r]")
    L, r, K = A.shape
    N = B.shape[1]
    _shape(B, (L, N, r), "B")
    _shape(scaling, (L,), "scaling")
    nbytes = _lib.q8_lora_packed_bytes(L, N, K, r)
    if nbytes == 0:
        raise Q8Error(Q8_ERR_SHAPE, "q8_lora_packed_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=A.device)
    _check(_lib.q8_lora_pack(A.data_ptr(), B.data_ptr(), scaling.data_ptr(), _DTYPE[A.dtype], L, r, N, K,
                             buf.data_ptr(), nbytes, _stream(A)), "q8_lora_pack")
    return PackedLora(buf, L, N, K, r, A.dtype)


@functools.lru_cache(maxsize=4096)
def _lora_space(M: int, K: int, L: int, r: int, device: int) -> int:
    with torch.cuda.device(device):
        return _lib.q8_linear_lora_workspace_bytes(M, K, L, r)


def linear_lora(x, input_scale, input_zero_point, packed: PackedTileWeight, weight_scales, bias,
                lora: PackedLora, adapter_ids, output_scale, output_zero_point,
                activation="none", out_dtype=torch.int8, out=None, workspace=None):
    """int8 x [M, K] times a shared int8 weight [N, K], plus each row's
    low-rank adapter (see q8_linear_lora): adapter_ids int32 [M], ids outside
    [0, L) for none; weight_scales and bias float32 [N]; out [M, N]."""
    at = _arg(x, torch.int8, "x")
    N, K = packed.N, packed.K
    if packed.E != 1:
        raise ValueError(f"the packed weight has {packed.E} groups, the shared projection one")
    if (lora.N, lora.K) != (N, K):
        raise ValueError(f"adapters are for {lora.N}x{lora.K}, the weight is {N}x{K}")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M, {K}], got {tuple(x.shape)}")
    M = x.shape[0]
    _need(weight_scales, torch.float32, "weight_scales")
    scales = _vector_arg(weight_scales, (N,), "weight_scales")
    b = _vector_arg(bias, (N,), "bias")
    ids = _arg(adapter_ids, torch.int32, "adapter_ids")
    _shape(adapter_ids, (M,), "adapter_ids")
    code = _out_code(out_dtype)
    out = _out(out, (M, N), out_dtype, x.device)
    nbytes = _lora_space(M, K, lora.L, lora.r, x.get_device())
    ws = _space(nbytes, x.device, workspace)
    _check(_lib.q8_linear_lora(
        at, M, K, float(input_scale), int(input_zero_point), packed.data.data_ptr(), N, scales, b,
        lora.data.data_ptr(), _DTYPE[lora.dtype], lora.L, lora.r, ids, float(output_scale),
        int(output_zero_point), activation.encode(), code, out.data_ptr(), ws.data_ptr(), nbytes,
        _stream(x)), "q8_linear_lora")
    return out
