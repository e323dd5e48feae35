"""Rows with a scale for each token (the last part of include/q8ta.h):
activations quantized as they come, the int8 products and the gated pair of
projections on them, and the gradients through int8 weights.

Argument marshalling only, like the rest of the package (the common case of it in
csrc/torch_calls.cpp); imported by it.  The products take float rows, which they
quantize, or int8 rows with their scales.  Float rows that require a gradient
get it where the transposed weight is given: the call is then recorded for
autograd, and keeps the int8 rows and their scales (linear_gated) or its output
under relu (linear_per_token), never the float rows.
"""
from __future__ import annotations

import dataclasses
import functools
import warnings
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import Q8_ERR_SHAPE, Q8Error, _check, _lib, _need, _stream
from .rows import _DTYPE, PackedTileWeight, _dtype_code, _shape, _space

_HALVES = (torch.float16, torch.bfloat16)


# A call for few tokens takes some 3 to 15 us on the GPU, so the host's part
# counts.  Calls as most are made (results and workspace from torch's allocator,
# nothing recorded) go through _torch_calls, which answers None where a tensor is
# not as it should be, and the status where the library refuses; then, and for
# all other calls, each argument is checked here by name.

class _Calls:
    def __getattr__(self, name):
        try:
            from . import _torch_calls
            f = getattr(_torch_calls, name)
        except ImportError as e:    # missing, or of another torch: the same kernels, later launched
            if not self.__dict__:
                warnings.warn(f"_torch_calls.so is not usable ({e}): calls take some 7 us longer on the "
                              "host until `python -m int8_quantized_q8ta_gb300._build --force`",
                              RuntimeWarning, stacklevel=3)
            f = _not_taken
        setattr(self, name, f)       # found here from the next call on
        return f


def _not_taken(*args) -> None:
    return None


_calls = _Calls()


def _done(result) -> bool:
    return result is not None and result.__class__ is not int


def _float_code(dtype, name: str) -> int:
    code = _DTYPE.get(dtype)
    if code is None or code == 3:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return code


def _at(t: torch.Tensor, dtype, shape, device: int, name: str) -> int:
    """The address of a contiguous tensor of this dtype and shape on a CUDA device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == device and t.is_contiguous()):
        _need(t, dtype, name)
        _shape(t, shape, name)
        raise ValueError(f"{name} must be on the rows' device, got {t.device}")
    return t.data_ptr()


def _matrix(t: torch.Tensor, codes, name: str) -> Tuple[int, int, int, int, int]:
    """(dtype code, address, rows, columns, device) of a contiguous CUDA matrix
    of one of these types."""
    code = _dtype_code(t, name)
    if code not in codes:
        types = ", ".join(str(d)[6:] for d, c in _DTYPE.items() if c in codes)
        raise TypeError(f"{name} must be {types}, got {t.dtype}")
    if not (t.is_cuda and t.is_contiguous()):
        _need(t, t.dtype, name)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix, got {tuple(shape)}")
    return code, t.data_ptr(), shape[0], shape[1], t.get_device()


def _packed_at(packed, device: int, name: str) -> int:
    data = packed.data
    if data.get_device() != device:
        raise ValueError(f"{name} must be on the rows' device, got {data.device}")
    return data.data_ptr()


def _result(out: Optional[torch.Tensor], shape, dtype, like: torch.Tensor, device: int,
            name: str = "out") -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _at(out, dtype, shape, device, name)
    return out


def _written(*given) -> None:
    """Given outputs count as written in place: a graph that keeps one (relu's
    gradient reads the forward output) then refuses its backward pass."""
    for t in given:
        if t is not None and not t.is_inference():
            increment_version(t)


# (sizes depend on the device's SMs)
@functools.lru_cache(maxsize=4096)
def _bytes(query: str, a: int, b: int, c: int, device: int) -> int:
    with torch.cuda.device(device):
        return getattr(_lib, query)(a, b, c)


def _run(name: str, device: int, *args) -> None:
    """One call of the library, with the tensors' device current: it asks the
    current one for its SMs, and launches there."""
    f = getattr(_lib, name)
    if device == torch.cuda.current_device():
        st = f(*args)
    else:
        with torch.cuda.device(device):
            st = f(*args)
    if st:
        _check(st, name)


def _workspace_at(nbytes: int, workspace, like: torch.Tensor, device: int):
    """(the workspace, to be kept until the launch, its address); some sizes need none."""
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    else:
        _space(nbytes, like.device, workspace)
        if workspace.get_device() != device:
            raise ValueError(f"workspace must be on the rows' device, got {workspace.device}")
    return workspace, workspace.data_ptr()


def _unfollowed(**tensors) -> None:
    """Refuses tensors that autograd follows where nothing is recorded."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} gets no gradient here: pass it detached")
        if forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{name} has a forward-mode tangent, which would be lost: pass it without")


def quantize_per_token(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                       scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Float rows [M, K] to int8, each with its own scale (see
    q8_quantize_per_token): returns (q int8 [M, K], scales float32 [M]).  Not
    recorded for autograd: x that requires a gradient is refused (the products take
    such rows themselves)."""
    if out is None and scales is None:
        r = _calls.quantize_per_token(x)
        if _done(r):
            return r
    code, at, M, K, device = _matrix(x, (0, 1, 2), "x")
    _unfollowed(x=x)
    q = _result(out, (M, K), torch.int8, x, device)
    s = _result(scales, (M,), torch.float32, x, device, "scales")
    _run("q8_quantize_per_token", device, at, code, M, K, q.data_ptr(), s.data_ptr(), _stream(x))
    _written(out, scales)
    return q, s


def dequantize_per_token(q: torch.Tensor, scales: torch.Tensor, out_dtype=torch.float32,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8 rows [M, K] times their scales, in a float type."""
    if out is None:
        r = _calls.dequantize_per_token(q, scales, out_dtype)
        if _done(r):
            return r
    _, at, M, K, device = _matrix(q, (3,), "q")
    s = _at(scales, torch.float32, (M,), device, "scales")
    _unfollowed(scales=scales)
    code = _float_code(out_dtype, "out_dtype")
    x = _result(out, (M, K), out_dtype, q, device)
    _run("q8_dequantize_per_token", device, at, s, M, K, code, x.data_ptr(), _stream(q))
    _written(out)
    return x


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


def _recorded(x, x_scales, weight_scales, bias, packed_t, out_dtype) -> bool:
    """Whether this call is recorded; what cannot be differentiated is refused."""
    _unfollowed(x_scales=x_scales, weight_scales=weight_scales, bias=bias)
    if not (x.requires_grad and torch.is_grad_enabled()):
        _unfollowed(x=x)
        return False
    if packed_t is None:
        raise ValueError("x requires a gradient: give packed_t, or pass x detached")
    if out_dtype not in _HALVES:
        raise TypeError("gradients are float16 or bfloat16: x requires one and out_dtype is "
                        f"{out_dtype}")
    return True


def _no_leaf(out: torch.Tensor) -> None:
    if out.requires_grad and out.is_leaf:
        raise ValueError("out is a leaf that requires a gradient: a result would overwrite it")


def _anew(out: torch.Tensor) -> torch.Tensor:
    """A given output that was the result of another recorded call (a buffer that
    each step of a training loop writes) holds nothing of it any more: it leaves that
    step's graph, whose backward pass has freed what it kept.  (A view stays part of
    its base, whose other rows may have a history that counts.)"""
    if out.requires_grad and not out._is_view():
        out.detach_()
    return out


def _rows(x, x_scales, K: int) -> Tuple[int, int, int, int, int]:
    """(dtype code, address, M, address of the scales, device) of either form of rows."""
    code, at, M, k, device = _matrix(x, (0, 1, 2, 3), "x")
    if k != K:
        raise ValueError(f"x must be [M, {K}], got {tuple(x.shape)}")
    if code == 3:
        if x_scales is None:
            raise ValueError("int8 x comes with x_scales")
        return code, at, M, _at(x_scales, torch.float32, (M,), device, "x_scales"), device
    if x_scales is not None:
        raise ValueError("float x is quantized here: x_scales must be None")
    return code, at, M, 0, device


def _out_dtype(x, out_dtype):
    if out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype is torch.int8 else x.dtype
    return out_dtype, _float_code(out_dtype, "out_dtype")


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
    if packed_t is not None and (packed_t.E, packed_t.N, packed_t.K) != (1, K, N):
        raise ValueError(f"packed_t must be of a {K}x{N} weight")
    if out is None and workspace is None:
        r = _calls.linear_per_token(x, x_scales, packed.data, N, K, weight_scales, bias, activation,
                                    out_dtype)
        if _done(r):
            return r
    code, at, M, s, device = _rows(x, x_scales, K)
    w = _packed_at(packed, device, "packed")
    scales = _at(weight_scales, torch.float32, (N,), device, "weight_scales")
    b = 0 if bias is None else _at(bias, torch.float32, (N,), device, "bias")
    out_dtype, out_code = _out_dtype(x, out_dtype)
    record = _recorded(x, x_scales, weight_scales, bias, packed_t, out_dtype)
    out = _result(out, (M, N), out_dtype, x, device)
    if record:
        _no_leaf(out)
    nbytes = _bytes("q8_linear_per_token_workspace_bytes", M, K, N, device)
    workspace, ws = _workspace_at(nbytes, workspace, x, device)
    _run("q8_linear_per_token", device, at, code, M, K, 0, s, w, N, scales, b, activation.encode(),
         out_code, out.data_ptr(), ws, nbytes, _stream(x))
    _written(out)
    if record:
        out = _Linear.apply(x, _anew(out), packed_t, weight_scales, activation == "relu")
    return out


def linear_per_token_backward(dy, packed_t: PackedTileWeight, weight_scales, y=None, out=None,
                              workspace=None):
    """The gradient of linear_per_token's rows (see
    q8_linear_per_token_backward): dy [M, N] float16 or bfloat16, y the forward
    output under relu; out [M, K] of dy's type."""
    K, N = packed_t.N, packed_t.K
    if packed_t.E != 1:
        raise ValueError(f"the packed weight has {packed_t.E} groups, this product takes one")
    if out is None and workspace is None:
        r = _calls.linear_per_token_backward(dy, packed_t.data, N, K, weight_scales, y)
        if _done(r):
            return r
    code, at, M, n, device = _matrix(dy, (1, 2), "dy")
    if n != N:
        raise ValueError(f"dy must be [M, {N}], got {tuple(dy.shape)}")
    y_at = 0 if y is None else _at(y, dy.dtype, (M, N), device, "y")
    w = _packed_at(packed_t, device, "packed_t")
    scales = _at(weight_scales, torch.float32, (N,), device, "weight_scales")
    out = _result(out, (M, K), dy.dtype, dy, device)
    nbytes = _bytes("q8_linear_per_token_backward_workspace_bytes", M, N, K, device)
    workspace, ws = _workspace_at(nbytes, workspace, dy, device)
    _run("q8_linear_per_token_backward", device, at, code, M, N, y_at, w, K, scales, out.data_ptr(),
         ws, nbytes, _stream(dy))
    _written(out)
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
    device = gate.get_device()
    if up.get_device() != device:
        raise ValueError(f"up must be on gate's device, got {up.device}")
    N, K = gate.shape
    nbytes = _lib.q8_gated_packed_weight_bytes(N, K, int(transposed))
    if nbytes == 0:
        raise Q8Error(Q8_ERR_SHAPE, "q8_gated_packed_weight_bytes")
    buf = torch.empty(nbytes, dtype=torch.uint8, device=gate.device)
    _run("q8_gated_pack_weight", device, gate.data_ptr(), up.data_ptr(), N, K, int(transposed),
         buf.data_ptr(), nbytes, _stream(gate))
    return PackedGatedWeight(buf, N, K, transposed)


def pack_gated_weight(gate: torch.Tensor, up: torch.Tensor) -> PackedGatedWeight:
    """Pack a gated pair's int8 weights [N, K] once, for linear_gated."""
    return _pack_gated(gate, up, False)


def pack_gated_weight_t(gate: torch.Tensor, up: torch.Tensor) -> PackedGatedWeight:
    """The same weights once more, transposed, for their gradient."""
    return _pack_gated(gate, up, True)


def _gated_pair(packed, packed_t) -> Tuple[int, int]:
    """(N, K) of a pair's weights, which packed_t, where given, has too."""
    if packed.transposed:
        raise ValueError("packed is a transposed weight (pack_gated_weight_t)")
    N, K = packed.N, packed.K
    if packed_t is not None and (not packed_t.transposed or (packed_t.N, packed_t.K) != (N, K)):
        raise ValueError(f"packed_t must come from pack_gated_weight_t of {N}x{K} weights")
    return N, K


def _gated_args(packed, weight_scales, bias, device: int) -> Tuple[int, int, int]:
    """The addresses of the pair's weights, scales and biases."""
    N = packed.N
    return (_packed_at(packed, device, "packed"),
            _at(weight_scales, torch.float32, (2, N), device, "weight_scales"),
            0 if bias is None else _at(bias, torch.float32, (2, N), device, "bias"))


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
    N, K = _gated_pair(packed, packed_t)
    if out is None and workspace is None:
        r = _calls.linear_gated(x, x_scales, packed.data, N, K, weight_scales, bias, activation,
                                out_dtype)
        if _done(r):
            return r
    code, at, M, s, device = _rows(x, x_scales, K)
    w, scales, b = _gated_args(packed, weight_scales, bias, device)
    out_dtype, out_code = _out_dtype(x, out_dtype)
    record = _recorded(x, x_scales, weight_scales, bias, packed_t, out_dtype)
    out = _result(out, (M, N), out_dtype, x, device)
    if record:
        _no_leaf(out)
    nbytes = _bytes("q8_linear_gated_workspace_bytes", M, K, N, device)
    workspace, ws = _workspace_at(nbytes, workspace, x, device)
    q_at = 0
    if record:
        x_q = torch.empty((M, K), dtype=torch.int8, device=x.device)
        x_scales = torch.empty(M, dtype=torch.float32, device=x.device)
        q_at, s = x_q.data_ptr(), x_scales.data_ptr()
    _run("q8_linear_gated", device, at, code, M, K, q_at, s, w, N, scales, b, activation.encode(),
         out_code, out.data_ptr(), ws, nbytes, _stream(x))
    _written(out)
    if record:
        out = _Gated.apply(x, _anew(out), x_q, x_scales, packed, packed_t, weight_scales, bias,
                           activation)
    return out


def linear_gated_backward(dh, x, x_scales, packed: PackedGatedWeight, packed_t: PackedGatedWeight,
                          weight_scales, bias, activation="silu", out=None, workspace=None):
    """The gradient of linear_gated's rows from the int8 rows x [M, K] and their
    scales (see q8_linear_gated_backward): dh [M, N] float16 or bfloat16; out
    [M, K] of dh's type."""
    if packed_t is None:
        raise ValueError("the gradient needs packed_t (pack_gated_weight_t)")
    N, K = _gated_pair(packed, packed_t)
    if out is None and workspace is None:
        r = _calls.linear_gated_backward(dh, x, x_scales, packed.data, packed_t.data, N, K,
                                         weight_scales, bias, activation)
        if _done(r):
            return r
    code, at, M, n, device = _matrix(dh, (1, 2), "dh")
    w, scales, b = _gated_args(packed, weight_scales, bias, device)
    if n != N:
        raise ValueError(f"dh must be [M, {N}], got {tuple(dh.shape)}")
    w_t = _packed_at(packed_t, device, "packed_t")
    q = _at(x, torch.int8, (M, K), device, "x")
    s = _at(x_scales, torch.float32, (M,), device, "x_scales")
    out = _result(out, (M, K), dh.dtype, dh, device)
    nbytes = _bytes("q8_linear_gated_backward_workspace_bytes", M, K, N, device)
    workspace, ws = _workspace_at(nbytes, workspace, dh, device)
    _run("q8_linear_gated_backward", device, at, code, M, N, q, s, K, w, w_t, scales, b,
         activation.encode(), out.data_ptr(), ws, nbytes, _stream(dh))
    _written(out)
    return out
