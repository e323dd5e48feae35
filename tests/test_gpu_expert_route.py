"""Tokens sorted by expert and back: sort, gather, combine and the gradients
against plain implementations in 64 bits.

Bounds, derived from the arithmetic and not from runs: a sum of k products in
f32 is within (k + 1) * 2^-23 * sum |w z| of the exact one (each product and
each addition rounds once, at most 2^-24 relative), and rounding to the row
type adds u * |y| (u = 2^-24, 2^-11, 2^-8 for f32, f16, bf16; f16 values below
2^-14 round to multiples of 2^-24).  A dot over H elements in any order is
within (H + 1) * 2^-23 * sum |dy z|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
DEV = torch.device("cuda:0")

UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOATS = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert q8.device_error(clear=True) == 0


def _ids(seed, T, k, E, drop=0.0, distinct=True):
    rng = np.random.default_rng(seed)
    if distinct and k <= E:
        ids = np.argsort(rng.random((T, E)) + 0.3 * rng.random(E), axis=1)[:, :k] if T else \
            np.zeros((0, k), np.int64)
    else:
        ids = rng.integers(0, E, (T, k))
    ids = ids.astype(np.int32)
    if drop:
        gone = rng.random((T, k)) < drop
        ids[gone] = rng.choice([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1], size=int(gone.sum()))
    return ids


def _sorted(ids, E):
    """Counting by hand: (order, position, offsets)."""
    flat = ids.reshape(-1).astype(np.int64)
    lists = [[] for _ in range(E)]
    for f, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(f)
    offsets = np.cumsum([0] + [len(a) for a in lists]).astype(np.int32)
    order = np.full(flat.size, -1, np.int32)
    position = np.full(flat.size, -1, np.int32)
    row = 0
    for a in lists:
        for f in a:
            order[row], position[f] = f, row
            row += 1
    return order, position.reshape(ids.shape), offsets


def _rand(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


SORTS = [(1, 1, 1, 0), (1, 8, 64, 0), (7, 3, 5, 0.3), (33, 1, 2, 0), (300, 8, 1024, 0.1),
         (513, 2, 1000, 0), (1000, 5, 17, 0.2), (5000, 4, 3, 0), (9000, 8, 128, 0.05),
         (40000, 3, 64, 0.0), (64, 6, 8, 1.0)]


@pytest.mark.parametrize("T,k,E,drop", SORTS)
def test_sort_is_the_stable_sort(T, k, E, drop):
    ids = _ids(T + k + E, T, k, E, drop)
    route = q8.expert_sort(torch.from_numpy(ids).to(DEV), E)
    order, position, offsets = _sorted(ids, E)
    np.testing.assert_array_equal(route.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(route.position.cpu().numpy(), position)
    np.testing.assert_array_equal(route.order.cpu().numpy(), order)


def test_sort_with_one_expert_taking_every_slot():
    ids = np.full((3000, 4), 2, np.int32)     # every lane of every warp holds the same id
    route = q8.expert_sort(torch.from_numpy(ids).to(DEV), 9)
    np.testing.assert_array_equal(route.order.cpu().numpy(), np.arange(12000))
    assert route.offsets.cpu().tolist() == [0, 0, 0] + [12000] * 7


def test_no_tokens():
    ids = torch.zeros((0, 4), dtype=torch.int32, device=DEV)
    x = torch.zeros((0, 16), device=DEV)
    rows, route = q8.expert_dispatch(x, ids, 6)
    assert rows.shape == (0, 16) and route.offsets.cpu().tolist() == [0] * 7
    w = torch.zeros((0, 4), device=DEV)
    assert q8.expert_combine(rows, w, route).shape == (0, 16)
    assert q8.expert_gather_backward(rows, route).shape == (0, 16)
    dz, dw = q8.expert_combine_backward(x, rows, w, route)
    assert dz.shape == (0, 16) and dw.shape == (0, 4)


# T, k, E, H, drop: one token, rows of one element, rows whose bytes are not a
# multiple of 16 (or of 4), rows longer than a warp's segment, dropped slots
SIZES = [(1, 1, 1, 1, 0), (1, 8, 64, 4096, 0), (5, 2, 4, 3, 0.4), (64, 4, 16, 257, 0),
         (130, 3, 7, 1003, 0.2), (77, 5, 31, 520, 0.1), (600, 8, 100, 1024, 0), (9, 4, 4, 8200, 0.5),
         (31, 2, 5, 64, 1.0)]


@pytest.mark.parametrize("dtype", FLOATS + [torch.int8])
@pytest.mark.parametrize("T,k,E,H,drop", SIZES)
def test_gather_copies_rows(T, k, E, H, drop, dtype):
    ids = _ids(3 * T + H, T, k, E, drop)
    x = _rand(H, (T, H), torch.float32)
    x = (x * 50).round().clamp(-128, 127).to(torch.int8) if dtype == torch.int8 else x.to(dtype)
    # what the tail held before must not survive
    out = torch.full((T * k, H), 77, dtype=dtype, device=DEV)
    rows, route = q8.expert_dispatch(x, torch.from_numpy(ids).to(DEV), E, out=out)
    order, _, offsets = _sorted(ids, E)
    ref = torch.zeros((T * k, H), dtype=dtype)
    n = offsets[-1]
    ref[:n] = x.cpu()[torch.from_numpy(order[:n].astype(np.int64)) // k]
    assert torch.equal(rows.cpu(), ref)
    again = q8.expert_gather(x, route)
    assert torch.equal(again.cpu(), ref)


def _slots(z, position):
    """float64 [T, k, H] rows of the kept slots, zeros elsewhere."""
    p = position.long()
    got = z.double().cpu()[p.clamp(min=0)]
    return torch.where((p >= 0)[:, :, None], got, torch.zeros((), dtype=torch.float64))


def _close(got, ref, bound):
    err = (got.double().cpu() - ref).abs()
    assert torch.all(err <= bound), float((err - bound).max())


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,k,E,H,drop", SIZES)
def test_combine_and_gradients(T, k, E, H, drop, dtype):
    ids = _ids(5 * T + H, T, k, E, drop)
    route = q8.expert_sort(torch.from_numpy(ids).to(DEV), E)
    position = route.position.cpu()
    z, dy = _rand(H + 1, (T * k, H), dtype), _rand(H + 2, (T, H), dtype)
    z[int(route.offsets[-1]):] = float("nan")      # rows of no slot are never read
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(T)).to(DEV)
    w64, dy64, zs = w.double().cpu(), dy.double().cpu(), _slots(z, position)
    u = UNIT[dtype]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0

    y = q8.expert_combine(z, w, route)
    ref = (w64[:, :, None] * zs).sum(1)
    size = (w64[:, :, None] * zs).abs().sum(1)
    _close(y, ref, u * ref.abs() + (k + 1) * 2.0 ** -23 * size + tiny)

    dx = q8.expert_gather_backward(z, route)
    ref = zs.sum(1)
    _close(dx, ref, u * ref.abs() + (k + 1) * 2.0 ** -23 * zs.abs().sum(1) + tiny)

    dz, dw = q8.expert_combine_backward(dy, z, w, route)
    ref = torch.zeros((T * k, H), dtype=torch.float64)
    kept = position >= 0
    ref[position[kept].long()] = (w64[:, :, None] * dy64[:, None, :])[kept]
    _close(dz, ref, (u + 2.0 ** -23) * ref.abs() + tiny)
    ref = (dy64[:, None, :] * zs).sum(2)
    _close(dw, ref, (H + 1) * 2.0 ** -23 * (dy64[:, None, :] * zs).abs().sum(2))
    assert torch.all(dw.cpu()[~kept] == 0)


@pytest.mark.parametrize("T,k", [(32, 8), (257, 1), (20, 8)])
def test_dispatch_around_one_launch_and_two(T, k):
    test_gather_copies_rows(T, k, 1024, 40, 0.1, torch.float16)
    test_gather_copies_rows(T, k, 9, 4100, 0.0, torch.int8)


@pytest.mark.parametrize("k", [31, 33, 70])
def test_more_slots_than_a_warp_has_lanes(k):
    test_combine_and_gradients(6, k, 80, 40, 0.2, torch.float32)
    test_combine_and_gradients(6, k, 80, 41, 0.2, torch.float16)


def test_gradients_against_differences():
    """<dy, combine> is linear in z and in w: a central difference along a
    direction equals the gradient's product with it, up to f32 rounding of
    the two values (2^-24 relative each, of sums of T*H terms)."""
    T, k, E, H = 24, 3, 6, 40
    ids = _ids(11, T, k, E, 0.1)
    route = q8.expert_sort(torch.from_numpy(ids).to(DEV), E)
    z, dy = _rand(1, (T * k, H), torch.float32), _rand(2, (T, H), torch.float32)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).to(DEV)
    dz, dw = q8.expert_combine_backward(dy, z, w, route)

    def value(z_, w_):
        return (dy.double() * q8.expert_combine(z_, w_, route).double()).sum()

    vz, vw = _rand(4, tuple(z.shape), torch.float32), _rand(5, tuple(w.shape), torch.float32)
    h = 0.25                                        # exact: a power of two, the function is linear
    size = (dy.abs().double().sum() * 4 * k)        # more than any |sum| of |w z| <= 4 on average
    for num, grad, v in (((value(z + h * vz, w) - value(z - h * vz, w)) / (2 * h), dz, vz),
                         ((value(z, w + h * vw) - value(z, w - h * vw)) / (2 * h), dw, vw)):
        got = (grad.double() * v.double()).sum()
        assert abs(float(num - got)) <= float(size) * (k + H) * 2.0 ** -23 / h


def test_gather_and_its_gradient_are_adjoint():
    T, k, E, H = 50, 4, 9, 33
    ids = _ids(12, T, k, E, 0.2)
    x, d = _rand(1, (T, H), torch.float32), _rand(2, (T * k, H), torch.float32)
    rows, route = q8.expert_dispatch(x, torch.from_numpy(ids).to(DEV), E)
    dx = q8.expert_gather_backward(d, route)
    a = (rows.double() * d.double()).sum()
    b = (x.double() * dx.double()).sum()
    size = (rows.double() * d.double()).abs().sum()
    assert abs(float(a - b)) <= float(size) * (k + 1) * 2.0 ** -23


def test_repeated_ids_in_a_token_and_special_values():
    """One token may name an expert twice; infinities and NaN of kept rows
    come through, those of dropped ones do not."""
    ids = torch.tensor([[1, 1], [0, -1]], dtype=torch.int32, device=DEV)
    route = q8.expert_sort(ids, 2)
    assert route.position.cpu().tolist() == [[1, 2], [0, -1]]
    z = torch.tensor([[1.0, 2.0], [float("inf"), 3.0], [1.0, float("nan")],
                      [float("nan")] * 2], device=DEV)
    w = torch.tensor([[0.5, 0.25], [2.0, float("inf")]], device=DEV)
    y = q8.expert_combine(z, w, route).cpu()
    assert y[0, 0] == float("inf") and torch.isnan(y[0, 1])
    assert y[1].tolist() == [2.0, 4.0]


def test_base_addresses_of_any_alignment():
    T, k, E, H = 40, 3, 8, 512
    ids = torch.from_numpy(_ids(13, T, k, E)).to(DEV)
    route = q8.expert_sort(ids, E)
    x = _rand(1, (T * H + 1,), torch.bfloat16)[1:].view(T, H)      # 2 bytes off
    out = torch.empty(T * k * H + 3, dtype=torch.bfloat16, device=DEV)[3:].view(T * k, H)
    rows = q8.expert_gather(x, route, out=out)
    order = route.order.long()
    assert torch.equal(rows, x[order // k])
    w = torch.ones((T, k), device=DEV)
    y = q8.expert_combine(rows, w, route)
    ref = x.double().cpu() * k
    _close(y, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -20 * ref.abs())


def test_other_stream():
    T, k, E, H = 256, 4, 16, 1024
    ids = torch.from_numpy(_ids(14, T, k, E)).to(DEV)
    x = _rand(1, (T, H), torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        rows, route = q8.expert_dispatch(x, ids, E)
        y = q8.expert_combine(rows, torch.ones((T, k), device=DEV), route)
    side.synchronize()
    assert torch.equal(y, x + x + x + x)


def test_captured_in_a_graph():
    T, k, E, H = 16, 4, 8, 256
    ids = torch.from_numpy(_ids(15, T, k, E)).to(DEV)
    x = _rand(1, (T, H), torch.float32)
    q8.expert_dispatch(x, ids, E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows, route = q8.expert_dispatch(x, ids, E)
    ids.copy_(torch.from_numpy(_ids(16, T, k, E)))
    graph.replay()
    torch.cuda.synchronize()
    order, position, offsets = _sorted(ids.cpu().numpy(), E)
    np.testing.assert_array_equal(route.order.cpu().numpy(), order)
    assert torch.equal(rows, x[torch.from_numpy(order).long().to(DEV) // k])


def test_binding_refusals():
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    x = torch.zeros((4, 8), device=DEV)
    route = q8.expert_sort(ids, 3)
    rows = torch.zeros((8, 8), device=DEV)
    w = torch.zeros((4, 2), device=DEV)
    with pytest.raises(TypeError):
        q8.expert_sort(ids.long(), 3)
    with pytest.raises(ValueError):
        q8.expert_sort(ids, 0)
    with pytest.raises(ValueError):
        q8.expert_sort(ids, 1025)
    with pytest.raises(ValueError):
        q8.expert_sort(ids.t(), 3)
    with pytest.raises(ValueError):
        q8.expert_gather(x[:3], route)
    with pytest.raises(TypeError):
        q8.expert_gather(x.double(), route)
    with pytest.raises(ValueError):
        q8.expert_combine(rows[:7], w, route)
    with pytest.raises(ValueError):
        q8.expert_combine(rows, w[:, :1].contiguous(), route)
    with pytest.raises(TypeError):
        q8.expert_combine(rows, w.half(), route)
    with pytest.raises(q8.Q8Error):
        q8.expert_combine(rows.to(torch.int8), w, route)
    with pytest.raises(TypeError):
        q8.expert_combine_backward(x.half(), rows, w, route)
    with pytest.raises(ValueError):
        q8.expert_gather_backward(rows.t(), route)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("fused", [False, True])
def test_gradients_through_autograd(dtype, fused):
    """dispatch, then combine: y = sum of the token's row times its kept slots'
    weights.  dz is w dy rounded once (u), dx the f32 sum of at most k of those
    rounded once, dw a dot over H elements."""
    T, k, E, H = 90, 4, 7, 72
    ids = torch.from_numpy(_ids(21, T, k, E, 0.2)).to(DEV)
    x = _rand(1, (T, H), dtype).requires_grad_()
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(4)).to(DEV).requires_grad_()
    if fused:
        rows, route = q8.expert_dispatch(x, ids, E)
    else:
        route = q8.expert_sort(ids, E)
        rows = q8.expert_gather(x, route)
    y = q8.expert_combine(rows, w, route)
    dy = _rand(2, (H, T), dtype).t()                  # not contiguous
    y.backward(dy)
    kept = (route.position >= 0).double().cpu()
    w64, x64, d64 = w.detach().double().cpu(), x.detach().double().cpu(), dy.double().cpu()
    u, tiny = UNIT[dtype], 2.0 ** -25 if dtype == torch.float16 else 0.0
    each = (w64 * kept)[:, :, None] * d64[:, None, :]
    size = each.abs().sum(1)
    _close(x.grad, each.sum(1), 2 * (u + 2.0 ** -23) * (1 + u) * size + (k + 1) * 2.0 ** -23 * size
           + (k + 1) * tiny)
    dot = x64 * d64
    ref = kept * dot.sum(1, keepdim=True)
    _close(w.grad, ref, (H + 1) * 2.0 ** -23 * kept * dot.abs().sum(1, keepdim=True))


def test_autograd_records_only_what_needs_it():
    T, k, E, H = 20, 2, 5, 16
    ids = torch.from_numpy(_ids(22, T, k, E)).to(DEV)
    x, w = _rand(1, (T, H), torch.float32), torch.full((T, k), 0.5, device=DEV)
    rows, route = q8.expert_dispatch(x, ids, E)
    y = q8.expert_combine(rows, w, route)
    assert not rows.requires_grad and not y.requires_grad
    w.requires_grad_()
    with torch.no_grad():
        assert not q8.expert_combine(rows, w, route).requires_grad
    out = torch.empty((T, H), device=DEV)
    got = q8.expert_combine(rows, w, route, out=out)   # the weights' gradient alone, and into out
    assert got is out and torch.equal(got, y)
    got.sum().backward()
    ref = x.double().sum(1).cpu()
    size = x.double().abs().sum(1).cpu()
    _close(w.grad, ref[:, None].expand(T, k), (H + 1) * 2.0 ** -23 * size[:, None])
    x.requires_grad_()
    kept = torch.empty((T * k, H), device=DEV)
    q8.expert_gather(x, route, out=kept)
    assert torch.equal(kept, rows) and kept.requires_grad
    (g,) = torch.autograd.grad(kept.sum(), x)
    assert torch.equal(g, torch.full_like(g, k))
