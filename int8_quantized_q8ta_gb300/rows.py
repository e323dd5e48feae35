"""Rows of one batch that go through different weights (the last part of
include/q8ta.h): tokens sorted by expert and back, with weights applied, and
the gradients.

Argument marshalling only, like the rest of the package; imported by it.
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Tuple

import torch

from . import Q8_ERR_SHAPE, Q8Error, _check, _lib, _need, _ptr, _stream, _workspace

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}


def _dtype_code(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16, bfloat16 or int8, got {t.dtype}")
    return code


def _shape(t: torch.Tensor, shape, name: str) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _out(out: Optional[torch.Tensor], shape, dtype, device, name: str = "out") -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, dtype, name)
    _shape(out, shape, name)
    return out


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


def _need_route(route: ExpertRoute) -> ExpertRoute:
    _need(route.order, torch.int32, "route.order")
    _need(route.position, torch.int32, "route.position")
    _need(route.offsets, torch.int32, "route.offsets")
    if route.position.dim() != 2 or route.offsets.dim() != 1 or route.E < 1:
        raise ValueError("route.position must be [T, k] and route.offsets [E + 1]")
    _shape(route.order, (route.T * route.k,), "route.order")
    return route


def _empty_route(expert_ids: torch.Tensor, num_experts: int) -> ExpertRoute:
    _need(expert_ids, torch.int32, "expert_ids")
    if expert_ids.dim() != 2:
        raise ValueError(f"expert_ids must be [T, k], got {tuple(expert_ids.shape)}")
    if not 1 <= num_experts <= 1024:
        raise ValueError(f"num_experts must lie in [1, 1024], got {num_experts}")
    # one allocation for the three parts, each of them contiguous
    T, k = expert_ids.shape
    R = T * k
    buf = torch.empty(2 * R + num_experts + 1, dtype=torch.int32, device=expert_ids.device)
    return ExpertRoute(buf[:R], buf[R:2 * R].view(T, k), buf[2 * R:])


def expert_sort(expert_ids: torch.Tensor, num_experts: int) -> ExpertRoute:
    """Slots of int32 expert_ids [T, k] sorted by expert, stable; ids outside
    [0, num_experts) are dropped slots."""
    route = _empty_route(expert_ids, num_experts)
    T, k = expert_ids.shape
    _check(_lib.q8_expert_sort(_ptr(expert_ids), T, k, num_experts, _ptr(route.order),
                               _ptr(route.position), _ptr(route.offsets), _stream(expert_ids)),
           "q8_expert_sort")
    return route


def expert_gather(x: torch.Tensor, route: ExpertRoute,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of x [T, H] (float32, float16, bfloat16 or int8) in sorted order,
    [T*k, H]; zeros from row offsets[E] on."""
    code = _dtype_code(x, "x")
    _need(x, x.dtype, "x")
    _need_route(route)
    T, k = route.T, route.k
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError(f"x must be [{T}, H], got {tuple(x.shape)}")
    H = x.shape[1]
    out = _out(out, (T * k, H), x.dtype, x.device)
    _check(_lib.q8_expert_gather(_ptr(x), code, T, k, H, route.E, _ptr(route.position),
                                 _ptr(route.offsets), _ptr(out), _stream(x)), "q8_expert_gather")
    return out


def expert_dispatch(x: torch.Tensor, expert_ids: torch.Tensor, num_experts: int,
                    out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ExpertRoute]:
    """expert_sort, then expert_gather: returns (rows, route)."""
    code = _dtype_code(x, "x")
    _need(x, x.dtype, "x")
    route = _empty_route(expert_ids, num_experts)
    T, k = expert_ids.shape
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError(f"x must be [{T}, H], got {tuple(x.shape)}")
    H = x.shape[1]
    out = _out(out, (T * k, H), x.dtype, x.device)
    _check(_lib.q8_expert_dispatch(_ptr(x), code, T, H, _ptr(expert_ids), k, num_experts,
                                   _ptr(route.order), _ptr(route.position), _ptr(route.offsets),
                                   _ptr(out), _stream(x)), "q8_expert_dispatch")
    return out, route


def _need_rows(t: torch.Tensor, route: ExpertRoute, name: str) -> int:
    code = _dtype_code(t, name)
    _need(t, t.dtype, name)
    if t.dim() != 2 or t.shape[0] != route.T * route.k:
        raise ValueError(f"{name} must be [{route.T * route.k}, H], got {tuple(t.shape)}")
    return code


def expert_gather_backward(d_rows: torch.Tensor, route: ExpertRoute,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gather's gradient: each token's kept rows added up in f32, [T, H]."""
    _need_route(route)
    code = _need_rows(d_rows, route, "d_rows")
    T, k, H = route.T, route.k, d_rows.shape[1]
    out = _out(out, (T, H), d_rows.dtype, d_rows.device)
    _check(_lib.q8_expert_gather_backward(_ptr(d_rows), code, T, k, H, _ptr(route.position),
                                          _ptr(out), _stream(d_rows)),
           "q8_expert_gather_backward")
    return out


def _need_weights(weights: torch.Tensor, route: ExpertRoute) -> None:
    _need(weights, torch.float32, "weights")
    _shape(weights, (route.T, route.k), "weights")


def expert_combine(z: torch.Tensor, weights: torch.Tensor, route: ExpertRoute,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * (slot (t, j)'s row of z), [T, H]."""
    _need_route(route)
    code = _need_rows(z, route, "z")
    _need_weights(weights, route)
    T, k, H = route.T, route.k, z.shape[1]
    out = _out(out, (T, H), z.dtype, z.device)
    _check(_lib.q8_expert_combine(_ptr(z), code, _ptr(weights), T, k, H, _ptr(route.position),
                                  _ptr(out), _stream(z)), "q8_expert_combine")
    return out


def expert_combine_backward(dy: torch.Tensor, z: torch.Tensor, weights: torch.Tensor,
                            route: ExpertRoute) -> Tuple[torch.Tensor, torch.Tensor]:
    """The combine's gradients (dz like z, dweights float32 [T, k])."""
    _need_route(route)
    code = _need_rows(z, route, "z")
    _need_weights(weights, route)
    _need(dy, z.dtype, "dy")
    T, k, H = route.T, route.k, z.shape[1]
    _shape(dy, (T, H), "dy")
    dz = torch.empty_like(z)
    dw = torch.empty((T, k), dtype=torch.float32, device=z.device)
    _check(_lib.q8_expert_combine_backward(_ptr(dy), _ptr(z), code, _ptr(weights), T, k, H,
                                           route.E, _ptr(route.position), _ptr(route.offsets),
                                           _ptr(dz), _ptr(dw), _stream(z)),
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
    _check(_lib.q8_tile_pack_weight(_ptr(weight), E, N, K, _ptr(buf), nbytes, _stream(weight)),
           "q8_tile_pack_weight")
    return PackedTileWeight(buf, E, N, K)


def linear_experts(x, input_scale, input_zero_point, packed: PackedTileWeight, weight_scales, bias,
                   route: ExpertRoute, output_scale, output_zero_point, activation="none",
                   x_sorted=False, out_dtype=torch.int8, out=None, workspace=None):
    """Sorted rows times the int8 weight of their expert (see
    q8_linear_experts): int8 x [T, K], or [T*k, K] in sorted order with
    ``x_sorted``; weight_scales and bias float32 [E, N]; out [T*k, N]."""
    _need(x, torch.int8, "x")
    _need_route(route)
    T, k, E, N = route.T, route.k, packed.E, packed.N
    if route.E != E:
        raise ValueError(f"the route has {route.E} experts, the packed weight {E}")
    _shape(x, (T * k if x_sorted else T, packed.K), "x")
    _need(weight_scales, torch.float32, "weight_scales")
    _shape(weight_scales, (E, N), "weight_scales")
    if bias is not None:
        _need(bias, torch.float32, "bias")
        _shape(bias, (E, N), "bias")
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype must be float32, float16, bfloat16 or int8, got {out_dtype}")
    out = _out(out, (T * k, N), out_dtype, x.device)
    nbytes = _lib.q8_linear_experts_workspace_bytes(T * k, packed.K, E)
    ws = _workspace(nbytes, x.device, workspace)
    _check(_lib.q8_linear_experts(
        _ptr(x), int(x_sorted), T, k, packed.K, float(input_scale), int(input_zero_point),
        _ptr(packed.data), E, N, _ptr(weight_scales), _ptr(bias), _ptr(route.order),
        _ptr(route.offsets), float(output_scale), int(output_zero_point), activation.encode(),
        _DTYPE[out_dtype], _ptr(out), _ptr(ws), nbytes, _stream(x)), "q8_linear_experts")
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
    scaling float32 [L] once."""
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
    _check(_lib.q8_lora_pack(_ptr(A), _ptr(B), _ptr(scaling), _DTYPE[A.dtype], L, r, N, K,
                             _ptr(buf), nbytes, _stream(A)), "q8_lora_pack")
    return PackedLora(buf, L, N, K, r, A.dtype)


def linear_lora(x, input_scale, input_zero_point, packed: PackedTileWeight, weight_scales, bias,
                lora: PackedLora, adapter_ids, output_scale, output_zero_point,
                activation="none", out_dtype=torch.int8, out=None, workspace=None):
    """int8 x [M, K] times a shared int8 weight [N, K], plus each row's
    low-rank adapter (see q8_linear_lora): adapter_ids int32 [M], ids outside
    [0, L) for none; weight_scales and bias float32 [N]; out [M, N]."""
    _need(x, torch.int8, "x")
    if packed.E != 1:
        raise ValueError(f"the packed weight has {packed.E} groups, the shared projection one")
    N, K = packed.N, packed.K
    if (lora.N, lora.K) != (N, K):
        raise ValueError(f"adapters are for {lora.N}x{lora.K}, the weight is {N}x{K}")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [M, {K}], got {tuple(x.shape)}")
    M = x.shape[0]
    _need(weight_scales, torch.float32, "weight_scales")
    _shape(weight_scales, (N,), "weight_scales")
    if bias is not None:
        _need(bias, torch.float32, "bias")
        _shape(bias, (N,), "bias")
    _need(adapter_ids, torch.int32, "adapter_ids")
    _shape(adapter_ids, (M,), "adapter_ids")
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype must be float32, float16, bfloat16 or int8, got {out_dtype}")
    out = _out(out, (M, N), out_dtype, x.device)
    nbytes = _lib.q8_linear_lora_workspace_bytes(M, K, lora.L, lora.r)
    ws = _workspace(nbytes, x.device, workspace)
    _check(_lib.q8_linear_lora(
        _ptr(x), M, K, float(input_scale), int(input_zero_point), _ptr(packed.data), N,
        _ptr(weight_scales), _ptr(bias), _ptr(lora.data), _DTYPE[lora.dtype], lora.L, lora.r,
        _ptr(adapter_ids), float(output_scale), int(output_zero_point), activation.encode(),
        _DTYPE[out_dtype], _ptr(out), _ptr(ws), nbytes, _stream(x)), "q8_linear_lora")
    return out
