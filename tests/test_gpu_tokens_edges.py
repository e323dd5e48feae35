"""Rows with a scale for each token where they end, overflow or are recorded:
what the calls of tests/test_gpu_tokens.py leave open.
"""
import ctypes

import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
DEV = torch.device("cuda:0")
FLOATS = [torch.float32, torch.float16, torch.bfloat16]
CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert q8.device_error(clear=True) == 0


def rows(seed, M, K, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, K, generator=g) * (0.1 + torch.rand(M, 1, generator=g) * 3)).to(dtype)


def weights(seed, *shape):
    g = torch.Generator().manual_seed(seed + 1000)
    w = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
    ws = (0.5 + torch.rand(shape[:-1], generator=g)) / (73.0 * shape[-1] ** 0.5)
    return w, ws, torch.randn(shape[:-1], generator=g) * 0.3


def at_offset(t, off):
    """The same rows `off` elements behind an aligned address, NaN around them."""
    flat = torch.full((t.numel() + 32,), float("nan"), dtype=t.dtype, device=DEV)
    flat[off:off + t.numel()] = t.reshape(-1).to(DEV)
    return flat[off:off + t.numel()].view(t.shape)


# ---- the int8 rows that a product writes beside its operand -------------------

@pytest.mark.parametrize("M", [9, 400])
@pytest.mark.parametrize("K", [130, 1978, 1979, 1980, 1981, 1982, 1983, 1984, 1985, 3967, 3968, 7936, 11903])
def test_every_int8_row_is_written(M, K):
    # 31 lanes of a warp store, so lengths of which every item but the last
    # fills whole warps count; rows that begin on each element of a vector
    N, poison = 24, 99
    w, ws, _ = weights(K, N, K)
    packed, wsd = q8.pack_tile_weight(w.to(DEV)), ws.to(DEV)
    lib = q8.lib()
    need = lib.q8_linear_per_token_workspace_bytes(M, K, N)
    space = torch.empty(need, dtype=torch.uint8, device=DEV)
    for dtype in FLOATS:
        x = rows(M + K, M, K, dtype)
        want_q, want_s = ref.quantize(x)
        for off in range(8):
            xd = at_offset(x, off)
            got = torch.full((M * K + 32,), poison, dtype=torch.int8, device=DEV)
            at = (off * 3) % 16
            s = torch.full((M,), -1.0, device=DEV)
            y = torch.empty((M, N), device=DEV)
            st = lib.q8_linear_per_token(xd.data_ptr(), CODE[dtype], M, K, got.data_ptr() + at, s.data_ptr(),
                                         packed.data.data_ptr(), N, wsd.data_ptr(), 0, b"none", 0, y.data_ptr(),
                                         space.data_ptr(), need,
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
            assert st == q8.Q8_OK
            got = got.cpu()
            assert torch.equal(got[at:at + M * K].view(M, K), want_q), (dtype, off)
            assert bool((got[:at] == poison).all()) and bool((got[at + M * K:] == poison).all())
            assert torch.equal(s.cpu(), want_s)


@pytest.mark.parametrize("M,K,off", [(9, 1983, 0), (400, 1983, 0), (40, 1984, 3), (20, 3967, 1)])
def test_recorded_rows_of_lengths_that_fill_warps(M, K, off):
    # the gradient comes from the int8 rows that the forward pass kept
    N = 40
    w, ws, b = weights(M, 2, N, K)
    gate, gt = (f(w[0].to(DEV), w[1].to(DEV)) for f in (q8.pack_gated_weight, q8.pack_gated_weight_t))
    x = at_offset(rows(M, M, K, torch.bfloat16), off)
    # (what the allocator hands out next held these bytes)
    torch.full((M, K), 99, dtype=torch.int8, device=DEV)
    leaf = x.detach().requires_grad_()
    h = q8.linear_gated(leaf, None, gate, ws.to(DEV), b.to(DEV), packed_t=gt)
    dh = rows(K, M, N, torch.bfloat16).to(DEV)
    (dx,) = torch.autograd.grad(h, leaf, dh)
    q, s = q8.quantize_per_token(x)
    assert torch.equal(dx, q8.linear_gated_backward(dh, q, s, gate, gt, ws.to(DEV), b.to(DEV)))


# ---- rows that hold an infinity ------------------------------------------------

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,K", [(2, 256), (5, 256), (60, 256), (200, 131), (3, 31), (400, 64)])
def test_nothing_finite_comes_of_a_row_with_an_infinity(dtype, M, K):
    x = rows(M + K, M, K, dtype)
    x[0, K // 3], x[1, 0] = float("-inf"), float("inf")
    w, ws, b = weights(M, 2, 70, K)
    wd, ws, b = w.to(DEV), ws.to(DEV), b.to(DEV)
    lin, gate = q8.pack_tile_weight(wd[0]), q8.pack_gated_weight(wd[0], wd[1])
    ws0, b0 = ws[0].contiguous(), b[0].contiguous()
    q, s = q8.quantize_per_token(x.to(DEV))
    assert bool(s[:2].isinf().all()) and bool(s[2:].isfinite().all())
    assert not bool(q8.dequantize_per_token(q, s)[:2].isfinite().any())
    for act in ("none", "relu"):
        for rows_, xs in ((x.to(DEV), None), (q, s)):
            y = q8.linear_per_token(rows_, xs, lin, ws0, b0, activation=act, out_dtype=torch.float32)
            assert not bool(y[:2].isfinite().any()) and bool(y[2:].isfinite().all()), act
    for act in ("silu", "gelu", "relu"):
        for rows_, xs in ((x.to(DEV), None), (q, s)):
            h = q8.linear_gated(rows_, xs, gate, ws, b, activation=act, out_dtype=torch.float32)
            assert not bool(h[:2].isfinite().any()) and bool(h[2:].isfinite().all()), act


# ---- gradients at the ends of the type's range ------------------------------------

@pytest.mark.parametrize("M", [3, 90])
def test_gradients_of_the_largest_values(M):
    # every |dy| within a factor of two of bfloat16's largest; scales that bring
    # the gradient back into its range
    N, K = 120, 70
    g = torch.Generator().manual_seed(M)
    top = float(torch.finfo(torch.bfloat16).max)
    dy = ((0.5 + 0.5 * torch.rand(M, N, generator=g)) * top).bfloat16()
    dy = torch.where(torch.rand(M, N, generator=g) < 0.5, -dy, dy)
    dy[0, 0], dy[1, 1] = top, -top
    w, _, _ = weights(M, N, K)
    ws = torch.full((N,), 2.0 ** -16)
    want, bound = ref.linear_grad(dy, w, ws)
    dx = q8.linear_per_token_backward(dy.to(DEV), q8.pack_tile_weight(w.t().contiguous().to(DEV)), ws.to(DEV))
    assert bool(dx.isfinite().all())
    assert bool(((dx.cpu().double() - want).abs() <= bound).all())
    # a row that does hold an infinity has no finite gradient, its neighbours keep theirs
    dy[1, 5] = float("inf")
    bad = q8.linear_per_token_backward(dy.to(DEV), q8.pack_tile_weight(w.t().contiguous().to(DEV)), ws.to(DEV))
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(bad[keep], dx[keep]) and not bool(bad[1].isfinite().any())


@pytest.mark.parametrize("M", [3, 90])
def test_gradients_of_the_smallest_values(M):
    # rows of nothing but bfloat16's subnormal numbers; the sums are normal ones
    N, K = 120, 70
    g = torch.Generator().manual_seed(M)
    dy = (torch.randint(-127, 128, (M, N), generator=g).double() * 2.0 ** -133).bfloat16()
    dy[0], dy[1] = 0, dy[1].sign() * 2.0 ** -133       # nothing, and the least there is
    w, _, _ = weights(M, N, K)
    ws = torch.ones(N)
    want, bound = ref.linear_grad(dy, w, ws)
    dx = q8.linear_per_token_backward(dy.to(DEV), q8.pack_tile_weight(w.t().contiguous().to(DEV)), ws.to(DEV))
    assert float(want.abs().max()) > 2.0 ** -120
    assert bool(((dx.cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("M", [3, 90])
def test_gated_gradients_whose_bound_overflows(M):
    # the bound on a row's operand, of which the sums' own bound is a part, passes
    # f32; the values, some 2^13 below it, do not
    N, K = 40, 640
    g0 = torch.Generator().manual_seed(M)
    q = torch.randint(-127, 128, (M, K), generator=g0, dtype=torch.int8)
    w = torch.randint(-1, 2, (2, N, K), generator=g0, dtype=torch.int8)
    xs, ws = torch.full((M,), 2.0 ** -10), torch.ones(2, N)
    dh = (torch.rand(M, N, generator=g0) + 0.5).bfloat16() * 2.0 ** 116
    assert 2.0 ** 116 * 1.25 * (2.0 ** -10 * 2.0 ** 14 * K) > 2.0 ** 128
    g, u = (ref.product(q, xs, w[i], ws[i], None) for i in (0, 1))
    want, bound = ref.gated_grad(dh, g, u, w, ws, "silu", xs)
    packed, packed_t = (f(w[0].to(DEV), w[1].to(DEV)) for f in (q8.pack_gated_weight, q8.pack_gated_weight_t))
    dx = q8.linear_gated_backward(dh.to(DEV), q.to(DEV), xs.to(DEV), packed, packed_t, ws.to(DEV), None)
    assert bool(dx.isfinite().all())
    assert bool(((dx.cpu().double() - want).abs() <= bound).all())


# ---- gated gradients of rows of almost nothing ---------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [3, 90])
def test_gated_gradients_of_rows_of_almost_nothing(act, dtype, M):
    # g and u near the smallest numbers, dh above 1: a row's power of two alone,
    # times dh, would pass f32 (a padded token under a loss scale)
    N, K = 120, 64
    q, xs = ref.quantize(rows(M, M, K))
    xs = xs * 2.0 ** -(torch.arange(M) % 3 * 8 + 104)
    dh = (rows(M + 1, M, N) * 2.0 ** 10).to(dtype)
    w, ws, _ = weights(M, 2, N, K)
    g, u = (ref.product(q, xs, w[i], ws[i], None) for i in (0, 1))
    want, bound = ref.gated_grad(dh, g, u, w, ws, act, xs)
    packed, packed_t = (f(w[0].to(DEV), w[1].to(DEV)) for f in (q8.pack_gated_weight, q8.pack_gated_weight_t))
    dx = q8.linear_gated_backward(dh.to(DEV), q.to(DEV), xs.to(DEV), packed, packed_t, ws.to(DEV), None,
                                  activation=act)
    assert bool(dx.isfinite().all())
    assert bool(((dx.cpu().double() - want).abs() <= bound).all())
    # with a bias that makes them large again only the gate's part is small
    b = torch.stack([torch.zeros(N), torch.full((N,), 3.0)])
    g, u = (ref.product(q, xs, w[i], ws[i], b[i]) for i in (0, 1))
    want, bound = ref.gated_grad(dh, g, u, w, ws, act, xs, b)
    dx = q8.linear_gated_backward(dh.to(DEV), q.to(DEV), xs.to(DEV), packed, packed_t, ws.to(DEV), b.to(DEV),
                                  activation=act)
    off = (dx.cpu().double() - want).abs()
    # (f16 has an end; sums of a few thousand lie below it)
    assert bool((off <= bound).all())


# ---- sums beyond 32 bits ----------------------------------------------------------

@pytest.mark.parametrize("M,K", [(1, 131071), (1, 131072), (1, 140001), (3, 140000), (70, 140064)])
def test_sums_wrap_modulo_2_32(M, K):
    # every product 128 * 128: 131071 of them are the last that fit
    N = 20
    q = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((N, K), -128, dtype=torch.int8)
    w[3, :5] = 127
    y = q8.linear_per_token(q.to(DEV), torch.ones(M, device=DEV), q8.pack_tile_weight(w.to(DEV)),
                            torch.ones(N, device=DEV), None, out_dtype=torch.float32)
    acc = (q[:1].long() * w.long()).sum(1)     # of each row
    acc = (acc + 2 ** 31) % 2 ** 32 - 2 ** 31
    assert torch.equal(y.cpu(), acc.float().expand(M, N))


# ---- what is recorded, and what is refused -----------------------------------------

class Pair:
    def __init__(self, N=90, K=64, M=12):
        w, ws, b = weights(2, 2, N, K)
        wd = w.to(DEV)
        self.lin, self.gate = q8.pack_tile_weight(wd[0]), q8.pack_gated_weight(wd[0], wd[1])
        self.lt, self.gt = q8.pack_tile_weight(wd[0].t().contiguous()), q8.pack_gated_weight_t(wd[0], wd[1])
        self.ws, self.b = ws.to(DEV), b.to(DEV)
        self.ws0, self.b0 = self.ws[0].contiguous(), self.b[0].contiguous()
        self.x = rows(3, M, K, torch.bfloat16).to(DEV)
        self.q, self.s = q8.quantize_per_token(self.x)


@pytest.mark.parametrize("given", [False, True])
def test_no_gradient_is_lost_without_a_word(given):
    # with the outputs given too, which takes the calls another way
    p = Pair()
    leaf, scales = p.x.clone().requires_grad_(), p.s.clone().requires_grad_()
    def out(cols, dtype=torch.bfloat16):
        return dict(out=torch.empty((12, cols), dtype=dtype, device=DEV)) if given else {}
    calls = [("x", lambda: q8.quantize_per_token(leaf, **out(64, torch.int8))),
             ("scales", lambda: q8.dequantize_per_token(p.q, scales, out_dtype=torch.bfloat16, **out(64))),
             ("x_scales", lambda: q8.linear_per_token(p.q, scales, p.lin, p.ws0, None, **out(90))),
             ("x_scales", lambda: q8.linear_per_token(p.q, scales, p.lin, p.ws0, None, packed_t=p.lt, **out(90))),
             ("x_scales", lambda: q8.linear_gated(p.q, scales, p.gate, p.ws, None, **out(90))),
             ("x_scales", lambda: q8.linear_gated(p.q, scales, p.gate, p.ws, None, packed_t=p.gt, **out(90)))]
    for name, call in calls:
        with pytest.raises(ValueError, match=rf"^{name} gets no gradient"):
            call()
        with torch.no_grad():
            call()


@pytest.mark.parametrize("given", [False, True])
def test_forward_mode_tangents_are_refused(given):
    p = Pair()
    import torch.autograd.forward_ad as fwd
    def out(cols, dtype=torch.bfloat16):
        return dict(out=torch.empty((12, cols), dtype=dtype, device=DEV)) if given else {}
    with fwd.dual_level():
        x, s = fwd.make_dual(p.x, p.x), fwd.make_dual(p.s, p.s)
        ws, ws0 = fwd.make_dual(p.ws, p.ws), fwd.make_dual(p.ws0, p.ws0)
        for call in (lambda: q8.quantize_per_token(x, **out(64, torch.int8)),
                     lambda: q8.dequantize_per_token(p.q, s, out_dtype=torch.bfloat16, **out(64)),
                     lambda: q8.linear_per_token(x, None, p.lin, p.ws0, None, **out(90)),
                     lambda: q8.linear_per_token(p.q, s, p.lin, p.ws0, None, **out(90)),
                     lambda: q8.linear_per_token(p.q, p.s, p.lin, ws0, None, **out(90)),
                     lambda: q8.linear_gated(x, None, p.gate, p.ws, None, **out(90)),
                     lambda: q8.linear_gated(p.q, p.s, p.gate, ws, None, **out(90))):
            with pytest.raises(ValueError, match="tangent"):
                call()
        # tensors without one are as ever
        q8.linear_per_token(p.q, p.s, p.lin, p.ws0, None, **out(90))


# ---- given outputs, recorded ------------------------------------------------------

def test_a_given_output_is_recorded_again_and_again():
    # a training loop whose results go to the same buffer each step
    p = Pair()
    y, h = (torch.empty((12, 90), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dy = rows(9, 12, 90, torch.bfloat16).to(DEV)
    for step in range(3):
        x = (p.x * (step + 1)).requires_grad_()
        got = q8.linear_per_token(x, None, p.lin, p.ws0, p.b0, activation="relu", packed_t=p.lt, out=y)
        assert got is y and y.requires_grad
        y.backward(dy)
        fresh = (p.x * (step + 1)).requires_grad_()
        q8.linear_per_token(fresh, None, p.lin, p.ws0, p.b0, activation="relu", packed_t=p.lt).backward(dy)
        assert torch.equal(x.grad, fresh.grad)
        x, fresh = ((p.x * (step + 1)).requires_grad_() for _ in range(2))
        assert q8.linear_gated(x, None, p.gate, p.ws, p.b, packed_t=p.gt, out=h) is h
        h.backward(dy)
        q8.linear_gated(fresh, None, p.gate, p.ws, p.b, packed_t=p.gt).backward(dy)
        assert torch.equal(x.grad, fresh.grad)
    # a leaf of the caller's that requires a gradient is no place for a result
    leaf = torch.zeros((12, 90), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    for call in (lambda: q8.linear_per_token(p.x.clone().requires_grad_(), None, p.lin, p.ws0, None, packed_t=p.lt, out=leaf),
                 lambda: q8.linear_gated(p.x.clone().requires_grad_(), None, p.gate, p.ws, None, packed_t=p.gt, out=leaf)):
        with pytest.raises(ValueError, match="out is a leaf"):
            call()
        assert bool((leaf == 0).all())


def test_a_recorded_step_in_a_graph():
    # forward and backward captured together and replayed with other rows
    p = Pair()
    x = p.x.clone().requires_grad_()
    dy = rows(9, 12, 64, torch.bfloat16).to(DEV)
    w, ws, _ = weights(5, 64, 90)
    down, down_t = q8.pack_tile_weight(w.to(DEV)), q8.pack_tile_weight(w.t().contiguous().to(DEV))
    wsd = ws.to(DEV)

    def step(x):
        h = q8.linear_gated(x, None, p.gate, p.ws, p.b, packed_t=p.gt)
        y = q8.linear_per_token(h, None, down, wsd, None, activation="relu", packed_t=down_t)
        return (y.detach(),) + torch.autograd.grad(y, x, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(x)
    for seed in (1, 2):
        other = rows(seed, 12, 64, torch.bfloat16).to(DEV)
        with torch.no_grad():
            x.copy_(other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, step(other.clone().requires_grad_())))


# ---- given outputs, written over -------------------------------------------------

def test_a_saved_output_that_a_later_call_overwrites():
    # relu's gradient reads the forward output: overwritten since, it is refused
    p = Pair()
    other = p.x.flip(0).contiguous()
    big, bq, bs = torch.empty((12, 90), device=DEV), torch.empty_like(p.q), torch.empty_like(p.s)
    y = torch.empty((12, 90), dtype=torch.bfloat16, device=DEV)
    dy = rows(9, 12, 90, torch.bfloat16).to(DEV)
    for write in (lambda: q8.linear_per_token(other, None, p.lin, p.ws0, None, out=y),
                  lambda: q8.linear_gated(other, None, p.gate, p.ws, None, out=y)):
        x = p.x.clone().requires_grad_()
        q8.linear_per_token(x, None, p.lin, p.ws0, p.b0, activation="relu", packed_t=p.lt, out=y)
        with torch.no_grad():
            write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward(dy)
    for t, write in ((bq, lambda: q8.quantize_per_token(other, out=bq)),
                     (bs, lambda: q8.quantize_per_token(other, scales=bs)),
                     (p.x, lambda: q8.dequantize_per_token(p.q, p.s, out_dtype=torch.bfloat16, out=p.x)),
                     (p.x, lambda: q8.linear_per_token_backward(dy, p.lt, p.ws0, out=p.x)),
                     (p.x, lambda: q8.linear_gated_backward(dy, p.q, p.s, p.gate, p.gt, p.ws, None, out=p.x)),
                     (big, lambda: q8.linear_per_token(other, None, p.lin, p.ws0, None, out_dtype=torch.float32, out=big))):
        before = t._version
        write()
        assert t._version > before
    with torch.inference_mode():
        q8.linear_per_token(other, None, p.lin, p.ws0, None, out=torch.empty_like(y))


# ---- f32 outputs of the gate ----------------------------------------------------------

def test_silu_of_float32_outputs_keeps_32_bits():
    # act(g) * u, u = 1.  exp is within 2 units in the last place, its sum with 1
    # and the division half a unit each, the two products half a unit each: 4
    # units, 2^-21 of the value; below the normal numbers what they are apart.
    K, N = 64, 4001
    w = torch.zeros(2, N, K, dtype=torch.int8)
    b = torch.zeros(2, N)
    b[0], b[1] = torch.linspace(-100, 100, N), 1.0
    ws = torch.ones(2, N)
    packed = q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV))
    want = ref.act64(b[0], "silu")[0]
    for M in (1, 6, 40, 100):
        q = torch.ones(M, K, dtype=torch.int8, device=DEV)
        h = q8.linear_gated(q, torch.ones(M, device=DEV), packed, ws.to(DEV), b.to(DEV), out_dtype=torch.float32)
        off = (h.cpu().double() - want).abs()
        assert bool((off <= want.abs() * 2.0 ** -21 + 2.0 ** -126).all()), float((off / want.abs().clamp(min=1e-300)).max())


# ---- other threads -----------------------------------------------------------------------

def test_other_threads_run_while_a_call_waits():
    # a full launch queue makes a call wait for the GPU: it waits without the
    # interpreter's lock
    import threading
    import time
    p = Pair()
    calls = (lambda: q8.quantize_per_token(p.x), lambda: q8.linear_per_token(p.q, p.s, p.lin, p.ws0, None))
    for call in calls:
        call()
        torch.cuda.synchronize()
        ticks, done = [], threading.Event()

        def tick():
            while not done.is_set():
                ticks.append(time.perf_counter())
                time.sleep(0.001)
        other = threading.Thread(target=tick)
        other.start()
        try:
            torch.cuda._sleep(1_500_000_000)   # some 0.75 s at 2 GHz
            begin = time.perf_counter()
            longest = 0.0
            for _ in range(3000):
                t = time.perf_counter()
                call()
                longest = max(longest, time.perf_counter() - t)
            end = time.perf_counter()
        finally:
            done.set()
            other.join()
            torch.cuda.synchronize()
        if longest < 0.1:
            pytest.skip("the launch queue did not fill")
        gaps = [b - a for a, b in zip(ticks, ticks[1:]) if a < end and b > begin]
        assert max(gaps) < 0.5 * longest


def test_threads_with_streams_of_their_own():
    # allocations and launches of several threads run at the same time
    import threading
    problems = [(M, N, K) for M, N, K in ((1, 900, 512), (7, 300, 1003), (40, 260, 1983), (150, 500, 640))]
    failed = []

    def work(M, N, K):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                w, ws, b = weights(M, 2, N, K)
                wd, ws, b = w.to(DEV), ws.to(DEV), b.to(DEV)
                lin, gate = q8.pack_tile_weight(wd[0]), q8.pack_gated_weight(wd[0], wd[1])
                gt = q8.pack_gated_weight_t(wd[0], wd[1])
                ws0, b0 = ws[0].contiguous(), b[0].contiguous()
                x = rows(M, M, K, torch.bfloat16).to(DEV)
                dh = rows(M + 1, M, N, torch.bfloat16).to(DEV)

                def step():
                    q, s = q8.quantize_per_token(x)
                    return (q, s, q8.linear_per_token(x, None, lin, ws0, b0), q8.linear_gated(q, s, gate, ws, b),
                            q8.linear_gated_backward(dh, q, s, gate, gt, ws, b))
                want = step()
                stream.synchronize()
                for _ in range(100):
                    got = step()
                    if not all(torch.equal(a, c) for a, c in zip(got, want)):
                        failed.append((M, N, K))
                        return
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=p) for p in problems]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
