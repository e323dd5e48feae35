"""Rows with a scale for each token: the quantizer and its way back, the
products and the gated pair, and the gradients, against tests/token_reference.py.

The quantizer's integers and scales and the plain product's outputs are
compared bit for bit; the gated pair and the gradients within bounds derived
there.
"""
import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
DEV = torch.device("cuda:0")
FLOATS = [torch.float32, torch.float16, torch.bfloat16]
HALVES = [torch.float16, torch.bfloat16]


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert q8.device_error(clear=True) == 0


def rows(seed, M, K, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * (0.1 + torch.rand(M, 1, generator=g) * 3)
    return (x * torch.where(torch.rand(K, generator=g) < 0.02, 8.0, 1.0)).to(dtype)


def weights(seed, *shape, lo=-127, hi=127):
    g = torch.Generator().manual_seed(seed + 1000)
    w = torch.randint(lo, hi + 1, shape, generator=g, dtype=torch.int8)
    ws = (0.5 + torch.rand(shape[:-1], generator=g)) / (73.0 * shape[-1] ** 0.5)
    return w, ws, torch.randn(shape[:-1], generator=g) * 0.3


def same(got, want):
    """Bit for bit (NaN equal to NaN)."""
    got = got.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape
    if not got.is_floating_point():
        assert torch.equal(got, want)
        return
    ok = (got == want) | (got.isnan() & want.isnan())
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} differ"


def within(got, want, bound):
    """A value beyond the type's largest by half a step or more rounds to an
    infinity (float16: from 65520 on), so one is right where the value within
    its bound may reach that."""
    info = torch.finfo(got.dtype)
    first = info.max * (1 + info.eps / 4)     # half a step of the largest's binade: max = (2 - eps) 2^e
    got = got.cpu().double()
    reached = got.isinf() & (got.sign() == want.sign()) & (want.abs() + bound >= first)
    over = torch.where(reached, torch.zeros((), dtype=torch.float64), (got - want).abs() - bound)
    assert bool((over <= 0).all()), (
        f"{int((over > 0).sum())} of {over.numel()} out of bounds, the worst by {float(over.max()):.3g} "
        f"of {float(bound.reshape(-1)[over.argmax()]):.3g}")


# ---- the quantizer ----------------------------------------------------------

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7), (3, 64), (2, 4096), (5, 1003), (400, 136), (37, 1000),
                                 (2, 11008), (1, 40001), (1, 40960), (700, 33)])
def test_quantize(dtype, M, K):
    x = rows(M * K, M, K, dtype)
    q, s = q8.quantize_per_token(x.to(DEV))
    want_q, want_s = ref.quantize(x)
    same(s, want_s)
    same(q, want_q)
    for out in FLOATS:
        back = q8.dequantize_per_token(q, s, out_dtype=out)
        same(back, (want_q.float() * want_s[:, None]).to(out))


@pytest.mark.parametrize("dtype", FLOATS)
def test_quantize_is_the_per_tensor_op_of_each_row(dtype):
    x = rows(5, 6, 512, dtype)
    q, s = q8.quantize_per_token(x.to(DEV))
    for m in range(6):
        row = x[m].float().to(DEV)
        assert torch.equal(q8.quantize_per_tensor(row, float(s[m]), 0), q[m])


def test_quantize_ties_and_extremes():
    # a = 127 * 2^-3: s = 1/8 exactly, so x * 8 is exact and ties go to even
    k = torch.arange(-127 * 2, 127 * 2 + 1).float() / 2
    x = torch.stack([k / 8, -k / 8, k * 2.0 ** 100, k * 2.0 ** -118])
    q, s = q8.quantize_per_token(x.to(DEV))
    want = torch.round(k).to(torch.int8)
    same(q, torch.stack([want, -want, want, want]))
    same(s, torch.tensor([0.125, 0.125, 2.0 ** 100, 2.0 ** -118]))


def test_quantize_rows_without_a_scale():
    tiny = torch.finfo(torch.float32).tiny
    x = torch.zeros(6, 70)
    x[1, 3] = 2.0 ** -149
    x[2, 5] = tiny * 126          # its scale is below the normal numbers
    x[3, 6] = tiny * 127          # and this one the smallest of them
    x[4, 8] = 1.0
    q, s = q8.quantize_per_token(x.to(DEV))
    same(s, torch.tensor([0, 0, 0, tiny, 1 / 127, 0]))
    want = torch.zeros(6, 70, dtype=torch.int8)
    want[3, 6] = want[4, 8] = 127
    same(q, want)
    assert torch.equal(q8.dequantize_per_token(q, s).cpu()[:3], torch.zeros(3, 70))


@pytest.mark.parametrize("dtype", FLOATS)
def test_infinities_and_nan_stay_with_their_rows(dtype):
    x = rows(9, 5, 256, dtype)
    bad = x.clone()
    bad[1, 17], bad[3, 200], bad[3, 4] = float("inf"), float("nan"), float("-inf")
    q, s = q8.quantize_per_token(bad.to(DEV))
    want_q, want_s = ref.quantize(x)
    keep = [0, 2, 4]
    assert torch.equal(q.cpu()[keep], want_q[keep]) and torch.equal(s.cpu()[keep], want_s[keep])
    assert s[1].isinf() and s[3].isnan()
    w, ws, b = weights(9, 40, 256)
    y = q8.linear_per_token(bad.to(DEV), None, q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), b.to(DEV))
    same(y[keep], ref.product(want_q, want_s, w, ws, b).to(dtype)[keep])
    assert not bool(y[[1, 3]].isfinite().any())


def test_quantize_unaligned_and_given_outputs():
    x = rows(3, 20, 96)
    for dtype in FLOATS:
        flat = torch.zeros(20 * 96 + 1, dtype=dtype, device=DEV)
        flat[1:] = x.to(dtype).reshape(-1).to(DEV)
        out = torch.full((20 * 96 + 3,), 55, dtype=torch.int8, device=DEV)
        scales = torch.full((22,), -1.0, device=DEV)
        q, s = q8.quantize_per_token(flat[1:].view(20, 96), out=out[1:-2].view(20, 96), scales=scales[1:21])
        want_q, want_s = ref.quantize(x.to(dtype))
        same(q, want_q)
        same(s, want_s)
        assert out[0] == 55 and bool((out[-2:] == 55).all())
        assert scales[0] == -1 and scales[21] == -1
        back = torch.full((20 * 96 + 2,), 7.0, dtype=dtype, device=DEV)
        q8.dequantize_per_token(q, s, out_dtype=dtype, out=back[1:-1].view(20, 96))
        same(back[1:-1].view(20, 96), (want_q.float() * want_s[:, None]).to(dtype))
        assert back[0] == 7 and back[-1] == 7


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,K", [(700, 1003), (400, 4097), (305, 33), (2000, 9), (1500, 2), (320, 40000), (3, 40001),
                                 (400, 16385), (777, 1234)])
def test_rows_of_any_length(dtype, M, K):
    x = rows(M + K, M, K, dtype)
    want_q, want_s = ref.quantize(x)
    q, s = q8.quantize_per_token(x.to(DEV))
    same(q, want_q)
    same(s, want_s)
    for out in FLOATS:
        same(q8.dequantize_per_token(q, s, out_dtype=out), (want_q.float() * want_s[:, None]).to(out))
    # and as the product's operand
    w, ws, _ = weights(K, 40, K)
    same(q8.linear_per_token(x.to(DEV), None, q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), None, out_dtype=torch.float32),
         gpu_product(want_q, want_s, w, ws, None))


@pytest.mark.parametrize("M,K", [(20, 97), (400, 131), (320, 264)])
def test_rows_anywhere(M, K):
    # rows that begin on any element, int8 ones on any byte; the words around stay
    for dtype in FLOATS:
        x = rows(K, M, K, dtype)
        want_q, want_s = ref.quantize(x)
        for off in range(9):
            flat = torch.full((M * K + 20,), float("nan"), dtype=dtype, device=DEV)
            flat[off:off + M * K] = x.reshape(-1).to(DEV)
            out = torch.full((M * K + 20,), 55, dtype=torch.int8, device=DEV)
            at = (off * 5) % 16
            q, s = q8.quantize_per_token(flat[off:off + M * K].view(M, K), out=out[at:at + M * K].view(M, K))
            same(q, want_q)
            same(s, want_s)
            assert bool((out[:at] == 55).all()) and bool((out[at + M * K:] == 55).all())
            back = torch.full((M * K + 20,), 7.0, dtype=dtype, device=DEV)
            q8.dequantize_per_token(q, s, out_dtype=dtype, out=back[off:off + M * K].view(M, K))
            same(back[off:off + M * K].view(M, K), (want_q.float() * want_s[:, None]).to(dtype))
            assert bool((back[:off] == 7).all()) and bool((back[off + M * K:] == 7).all())


# ---- the product ------------------------------------------------------------

SIZES = [(1, 4, 1), (1, 128, 64), (1, 1000, 1234), (2, 260, 4096), (3, 37, 65), (8, 1003, 512), (16, 4100, 320),
         (17, 129, 2050), (33, 640, 1000), (64, 128, 4096), (65, 300, 130), (100, 4100, 200), (192, 256, 777),
         (193, 130, 640), (300, 1000, 1234), (777, 72, 100)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_int8_rows(M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    q = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8)
    xs = torch.rand(M, generator=g) * 0.05
    w, ws, b = weights(M + N, N, K, lo=-128)
    packed = q8.pack_tile_weight(w.to(DEV))
    for out, bias, act in ((torch.float32, b, "none"), (torch.bfloat16, None, "relu"),
                           (torch.float16, b, "relu")):
        y = q8.linear_per_token(q.to(DEV), xs.to(DEV), packed, ws.to(DEV), None if bias is None else b.to(DEV),
                                activation=act, out_dtype=out)
        v = ref.product(q, xs, w, ws, bias)
        same(y, (v.clamp(min=0) if act == "relu" else v).to(out))


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,N,K", [(1, 640, 4096), (4, 100, 1003), (16, 516, 256), (40, 200, 2000), (70, 129, 1000),
                                   (260, 140, 264)])
def test_linear_float_rows(dtype, M, N, K):
    x = rows(M + K, M, K, dtype)
    w, ws, b = weights(M + N, N, K)
    y = q8.linear_per_token(x.to(DEV), None, q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), b.to(DEV))
    same(y, ref.product(*ref.quantize(x), w, ws, b).to(dtype))


@pytest.mark.parametrize("M", [1, 5, 16, 33, 70])
def test_linear_sums_beyond_24_bits(M):
    # every product 127 * 127 or -128 * -128: sums far beyond f32's integers
    K, N = 9000, 130
    q = torch.full((M, K), 127, dtype=torch.int8)
    w = torch.full((N, K), 127, dtype=torch.int8)
    q[0], w[5] = -128, -128
    w[7, 1] = 126
    xs, ws = torch.ones(M), torch.ones(N)
    y = q8.linear_per_token(q.to(DEV), xs.to(DEV), q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), None,
                            out_dtype=torch.float32)
    same(y, ref.product(q, xs, w, ws, None))


def test_no_rows_and_rows_behind_the_last():
    w, ws, b = weights(1, 200, 96)
    packed, gate = q8.pack_tile_weight(w.to(DEV)), q8.pack_gated_weight(w.to(DEV), w.to(DEV))
    pt = q8.pack_tile_weight(w.t().contiguous().to(DEV))
    gt = q8.pack_gated_weight_t(w.to(DEV), w.to(DEV))
    ws, ws2 = ws.to(DEV), torch.stack([ws, ws]).to(DEV)
    none = torch.empty(0, 96, device=DEV, dtype=torch.bfloat16)
    dnone = torch.empty(0, 200, device=DEV, dtype=torch.bfloat16)
    q, s = q8.quantize_per_token(none)
    assert q.shape == (0, 96) and s.shape == (0,)
    assert q8.dequantize_per_token(q, s).shape == (0, 96)
    assert q8.linear_per_token(none, None, packed, ws, None).shape == (0, 200)
    assert q8.linear_gated(none, None, gate, ws2, None).shape == (0, 200)
    assert q8.linear_per_token_backward(dnone, pt, ws).shape == (0, 96)
    assert q8.linear_gated_backward(dnone, q, s, gate, gt, ws2, None).shape == (0, 96)
    for M in (1, 3, 20, 33, 66, 200):
        x = rows(M, M, 96, torch.bfloat16).to(DEV)
        dy = rows(M, M, 200, torch.bfloat16).to(DEV)
        big = torch.full((M + 2, 200), 7.0, device=DEV, dtype=torch.bfloat16)
        dbig = torch.full((M + 2, 96), 7.0, device=DEV, dtype=torch.bfloat16)
        q, s = q8.quantize_per_token(x)
        q8.linear_per_token(x, None, packed, ws, None, out=big[1:-1])
        assert bool((big[[0, -1]] == 7).all())
        q8.linear_gated(x, None, gate, ws2, None, out=big[1:-1])
        assert bool((big[[0, -1]] == 7).all())
        q8.linear_per_token_backward(dy, pt, ws, out=dbig[1:-1])
        assert bool((dbig[[0, -1]] == 7).all())
        q8.linear_gated_backward(dy, q, s, gate, gt, ws2, None, out=dbig[1:-1])
        assert bool((dbig[[0, -1]] == 7).all())


def test_dirty_workspaces():
    # what an earlier call left, NaN patterns among it, changes nothing
    for M in (1, 8, 40, 150):
        x = rows(M, M, 300, torch.float16)
        dh = rows(M + 1, M, 500, torch.float16).to(DEV)
        w, ws, b = weights(M, 2, 500, 300)
        lin, gate = q8.pack_tile_weight(w[0].to(DEV)), q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV))
        pt = q8.pack_tile_weight(w[0].t().contiguous().to(DEV))
        gt = q8.pack_gated_weight_t(w[0].to(DEV), w[1].to(DEV))
        ws, b, x = ws.to(DEV), b.to(DEV), x.to(DEV)
        q, s = q8.quantize_per_token(x)
        ws0, b0 = ws[0].contiguous(), b[0].contiguous()
        calls = [lambda w: q8.linear_per_token(x, None, lin, ws0, b0, workspace=w),
                 lambda w: q8.linear_gated(x, None, gate, ws, b, workspace=w),
                 lambda w: q8.linear_per_token_backward(dh, pt, ws0, workspace=w),
                 lambda w: q8.linear_gated_backward(dh, q, s, gate, gt, ws, b, workspace=w)]
        space = torch.empty(128 << 20, dtype=torch.uint8, device=DEV)
        for call in calls:
            want = call(None)
            for fill in (0xFF, 0x7F, 0):
                space.fill_(fill)
                assert torch.equal(call(space), want)


def gpu_product(q, xs, w, ws, b):
    """ref.product of sizes that the CPU would take long for (the sums are exact
    wherever they are computed)."""
    return ref.product(*(None if t is None else t.to(DEV) for t in (q, xs, w, ws, b))).cpu()


# Tiles of one group that fill the GPU once or more, with what is left from a few
# units to nearly a wave: whole units, units cut across runs, units shared.
@pytest.mark.parametrize("M,N,K", [(640, 1280, 4096), (900, 1280, 4096), (1300, 1280, 4096), (2000, 1280, 4096),
                                   (2048, 4096, 2816), (3000, 1280, 4096), (3700, 1280, 4096), (4096, 1280, 4096),
                                   (640, 2560, 3500), (600, 6000, 2500), (900, 4096, 4096), (100, 20000, 1000)])
def test_every_way_to_split_units(M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    q = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8)
    xs = torch.rand(M, generator=g) * 0.05
    w, ws, b = weights(M + N, N, K, lo=-128)
    y = q8.linear_per_token(q.to(DEV), xs.to(DEV), q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), b.to(DEV),
                            out_dtype=torch.float32)
    same(y, gpu_product(q, xs, w, ws, b))


@pytest.mark.parametrize("M,N,K", [(1, 6007, 700), (2, 9001, 333), (5, 9001, 640), (7, 4113, 4096), (1, 40, 100000),
                                   (2, 130, 70001), (8, 70, 4097), (6, 333, 5000), (9, 200, 4096)])
def test_few_rows_of_many_channels_or_inputs(M, N, K):
    dtype = FLOATS[(M + N + K) % 3]
    x = rows(M + K, M, K, dtype)
    w, ws, b = weights(M + N, N, K)
    qs = ref.quantize(x)
    want = gpu_product(*qs, w, ws, b)
    packed = q8.pack_tile_weight(w.to(DEV))
    same(q8.linear_per_token(x.to(DEV), None, packed, ws.to(DEV), b.to(DEV)), want.to(dtype))
    same(q8.linear_per_token(qs[0].to(DEV), qs[1].to(DEV), packed, ws.to(DEV), b.to(DEV), out_dtype=dtype),
         want.to(dtype))


@pytest.mark.parametrize("M,N,K", [(3, 2600, 21845), (3, 90, 21846), (4, 333, 11003), (5, 5000, 13104), (8, 700, 8192),
                                   (8, 130, 8193), (7, 200, 9361)])
def test_few_long_int8_rows(M, N, K):
    # up to 65536 values and just beyond; the rows' last bytes and the next one's first
    g = torch.Generator().manual_seed(M * K)
    q = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8)
    q[:, 0], q[:, -1] = 127, -128
    xs = torch.rand(M, generator=g) * 0.05
    w, ws, b = weights(M + N, N, K, lo=-128)
    packed = q8.pack_tile_weight(w.to(DEV))
    want = gpu_product(q, xs, w, ws, b)
    off = torch.zeros(M * K + 3, dtype=torch.int8, device=DEV)
    off[3:] = q.reshape(-1).to(DEV)
    for rows8 in (q.to(DEV), off[3:].view(M, K)):
        same(q8.linear_per_token(rows8, xs.to(DEV), packed, ws.to(DEV), b.to(DEV), out_dtype=torch.float32), want)


@pytest.mark.parametrize("M,K", [(1, 31), (3, 1003), (8, 517)])
def test_few_rows_anywhere(M, K):
    # rows that begin on any element, int8 ones on any byte; the words around stay
    w, ws, b = weights(M, 90, K)
    packed = q8.pack_tile_weight(w.to(DEV))
    for dtype in FLOATS:
        x = rows(K, M, K, dtype)
        qs = ref.quantize(x)
        want = ref.product(*qs, w, ws, b).to(dtype)
        for off in range(8):
            flat = torch.full((M * K + 16,), float("nan"), dtype=dtype, device=DEV)
            flat[off:off + M * K] = x.reshape(-1).to(DEV)
            same(q8.linear_per_token(flat[off:off + M * K].view(M, K), None, packed, ws.to(DEV), b.to(DEV)), want)
            ints = torch.full((M * K + 16,), 99, dtype=torch.int8, device=DEV)
            ints[off:off + M * K] = qs[0].reshape(-1).to(DEV)
            same(q8.linear_per_token(ints[off:off + M * K].view(M, K), qs[1].to(DEV), packed, ws.to(DEV), b.to(DEV),
                                     out_dtype=dtype), want)


# ---- the gated pair ---------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 5), (1, 100, 4096), (2, 16, 64), (5, 17, 1003), (8, 2749, 96), (16, 333, 512),
                                   (33, 130, 1031), (64, 2100, 128), (65, 63, 200), (150, 90, 400), (200, 2000, 72),
                                   (400, 31, 130)])
def test_gated(act, M, N, K):
    dtype = FLOATS[(M + N + K) % 3]
    x = rows(M + N, M, K, dtype)
    w, ws, b = weights(K, 2, N, K)
    b = b if M % 2 else None
    q, xs = ref.quantize(x)
    g, u = (ref.product(q, xs, w[i], ws[i], None if b is None else b[i]) for i in (0, 1))
    want, bound = ref.gated(g, u, act, dtype)
    packed = q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV))
    args = (packed, ws.to(DEV), None if b is None else b.to(DEV))
    h = q8.linear_gated(x.to(DEV), None, *args, activation=act)
    assert h.dtype == dtype
    within(h, want, bound)
    # int8 rows with their scales give the same
    assert torch.equal(q8.linear_gated(q.to(DEV), xs.to(DEV), *args, activation=act, out_dtype=dtype), h)


def test_gated_of_far_values():
    # gates from -200 to 200: the sigmoid runs into 0 and 1 without NaN
    K, N = 64, 401
    w = torch.zeros(2, N, K, dtype=torch.int8)
    w[:, :, 0] = 1
    ws = torch.ones(2, N)
    b = torch.zeros(2, N)
    b[0] = torch.arange(-200, 201).float()
    q = torch.ones(2, K, dtype=torch.int8)
    q[:, 0] = 0
    xs = torch.ones(2)
    for act in ("silu", "gelu", "relu"):
        b[1] = 1.0
        h = q8.linear_gated(q.to(DEV), xs.to(DEV), q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV)), ws.to(DEV),
                            b.to(DEV), activation=act, out_dtype=torch.float32)
        g = b[0].expand(2, N)
        want, bound = ref.gated(g, torch.ones(2, N), act, torch.float32)
        # (below 2^-126 the fast division gives 0)
        within(h, want, bound + 200 * 2.0 ** -126)


# ---- the gradients ----------------------------------------------------------

@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 512, 300), (3, 65, 129), (16, 1000, 256), (40, 333, 640),
                                   (64, 4096, 130), (65, 200, 300), (190, 1003, 72), (300, 130, 1234)])
def test_linear_gradient(dtype, relu, M, N, K):
    dy, y = rows(M + N, M, N, dtype), rows(M + K, M, N, dtype)
    w, ws, _ = weights(N, N, K, lo=-128)
    want, bound = ref.linear_grad(dy, w, ws, y if relu else None)
    packed_t = q8.pack_tile_weight(w.t().contiguous().to(DEV))
    dx = q8.linear_per_token_backward(dy.to(DEV), packed_t, ws.to(DEV), y=y.to(DEV) if relu else None)
    assert dx.dtype == dtype
    within(dx, want, bound)
    again = q8.linear_per_token_backward(dy.to(DEV), packed_t, ws.to(DEV), y=y.to(DEV) if relu else None)
    assert torch.equal(dx, again)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 2), (1, 300, 500), (7, 65, 100), (20, 1000, 64), (64, 140, 1100),
                                   (65, 72, 260), (130, 500, 140), (200, 129, 333)])
def test_gated_gradient(dtype, act, M, N, K):
    q, xs = ref.quantize(rows(M + K, M, K))
    dh = rows(M + N, M, N, dtype)
    w, ws, b = weights(N, 2, N, K, lo=-128)
    b = b if N % 2 else None
    g, u = (ref.product(q, xs, w[i], ws[i], None if b is None else b[i]) for i in (0, 1))
    want, bound = ref.gated_grad(dh, g, u, w, ws, act, xs, b)
    packed = q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV))
    packed_t = q8.pack_gated_weight_t(w[0].to(DEV), w[1].to(DEV))
    args = (dh.to(DEV), q.to(DEV), xs.to(DEV), packed, packed_t, ws.to(DEV), None if b is None else b.to(DEV))
    dx = q8.linear_gated_backward(*args, activation=act)
    assert dx.dtype == dtype
    within(dx, want, bound)
    assert torch.equal(dx, q8.linear_gated_backward(*args, activation=act))


@pytest.mark.parametrize("M,N,K", [(700, 131, 77), (1900, 6000, 2500), (1024, 8200, 1030), (400, 1003, 72)])
def test_gradients_of_many_rows(M, N, K):
    # bounds from 64-bit products on the GPU; rows that begin on any element
    dtype = HALVES[M % 2]
    dy, y = rows(M + N, M, N, dtype), rows(M + K, M, N, dtype)
    w, ws, b = weights(N, 2, N, K, lo=-128)
    q, xs = ref.quantize(rows(M, M, K))
    def far(t):
        flat = torch.full((t.numel() + 3,), float("nan"), dtype=t.dtype, device=DEV)
        flat[3:] = t.reshape(-1).to(DEV)
        return flat[3:].view(t.shape)
    dyd, yd, wd, wsd, bd, qd, xsd = (t.to(DEV) for t in (dy, y, w, ws, b, q, xs))
    masked = torch.where(yd > 0, dyd, torch.zeros((), dtype=dtype, device=DEV))
    packed_t = q8.pack_tile_weight(wd[0].t().contiguous())
    for relu in (False, True):
        want, bound = ref.linear_grad(masked if relu else dyd, wd[0], wsd[0])
        dx = q8.linear_per_token_backward(far(dy), packed_t, wsd[0].contiguous(), y=far(y) if relu else None)
        within(dx, want.cpu(), bound.cpu())
    g, u = (ref.product(qd, xsd, wd[i], wsd[i], bd[i]) for i in (0, 1))
    want, bound = ref.gated_grad(dyd, g, u, wd, wsd, "silu", xsd, bd)
    ints = torch.full((M * K + 5,), 99, dtype=torch.int8, device=DEV)
    ints[5:] = qd.reshape(-1)
    dx = q8.linear_gated_backward(far(dy), ints[5:].view(M, K), xsd, q8.pack_gated_weight(wd[0], wd[1]),
                                  q8.pack_gated_weight_t(wd[0], wd[1]), wsd, bd)
    within(dx, want.cpu(), bound.cpu())


@pytest.mark.parametrize("M,N,K", [(3, 65, 40), (100, 320, 96)])
@pytest.mark.parametrize("dtype", HALVES)
def test_masked_gradients_count_as_zeros(dtype, M, N, K):
    # whatever they are: infinities, NaN, the type's largest
    dy, y = rows(M, M, N, dtype), rows(K, M, N, dtype)
    y[0] = -1.0                                        # a row of nothing
    y[1, ::2], y[1, 1::2] = float("nan"), -0.0         # NaN and zeros are not above 0
    w, ws, _ = weights(N, N, K)
    packed_t = q8.pack_tile_weight(w.t().contiguous().to(DEV))
    clean = torch.where(y > 0, dy, torch.zeros((), dtype=dtype))
    want = q8.linear_per_token_backward(clean.to(DEV), packed_t, ws.to(DEV))
    for bad in (float("inf"), float("-inf"), float("nan"), torch.finfo(dtype).max):
        dirty = torch.where(y > 0, dy, torch.full((), bad, dtype=dtype))
        got = q8.linear_per_token_backward(dirty.to(DEV), packed_t, ws.to(DEV), y=y.to(DEV))
        assert torch.equal(got, want) and bool((got[:2] == 0).all())


def test_offsets_beyond_32_bits():
    # 2.2e9 values, 4.5 GB, of which the last rows count
    M, K, N = 700_001, 3201, 64
    w, ws, b = weights(3, N, K)
    last = rows(1, 40, K, torch.bfloat16)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[-40:] = last.to(DEV)
    want_q, want_s = ref.quantize(last)
    q, s = q8.quantize_per_token(x)
    same(q[-40:], want_q)
    same(s[-40:], want_s)
    same(q8.dequantize_per_token(q, s, out_dtype=torch.bfloat16, out=x)[-40:],
         (want_q.float() * want_s[:, None]).bfloat16())
    del x
    y = q8.linear_per_token(q, s, q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), b.to(DEV))
    same(y[-40:], ref.product(want_q, want_s, w, ws, b).bfloat16())
    # and 64 inputs to 3201 outputs, its gradient back, the gated pair's
    del q
    x = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    x[-40:] = rows(2, 40, N, torch.bfloat16).to(DEV)
    wt = w.t().contiguous()
    wts = torch.full((2, K), 0.01)
    y = q8.linear_per_token(x, None, q8.pack_tile_weight(wt.to(DEV)), wts[0].to(DEV), None)
    same(y[-40:], ref.product(*ref.quantize(x[-40:].cpu()), wt, wts[0], None).bfloat16())
    dx = q8.linear_per_token_backward(y, q8.pack_tile_weight(w.to(DEV)), wts[0].to(DEV))
    few = q8.linear_per_token_backward(y[-40:], q8.pack_tile_weight(w.to(DEV)), wts[0].to(DEV))
    want, bound = ref.linear_grad(y[-40:].cpu(), wt, wts[0])
    within(dx[-40:], want, bound)
    within(few, want, bound)
    q, s = q8.quantize_per_token(x)
    del dx, x
    pair = (wt.to(DEV), wt.to(DEV))
    gate, gt = q8.pack_gated_weight(*pair), q8.pack_gated_weight_t(*pair)
    dx = q8.linear_gated_backward(y, q, s, gate, gt, wts.to(DEV), None)
    g = ref.product(q[-40:].cpu(), s[-40:].cpu(), wt, wts[0], None)
    within(dx[-40:], *ref.gated_grad(y[-40:].cpu(), g, g, torch.stack([wt, wt]), wts, "silu", s[-40:].cpu()))
    h = q8.linear_gated(q, s, gate, wts.to(DEV), None, out=y)
    within(h[-40:], *ref.gated(g, g, "silu", torch.bfloat16))


@pytest.mark.parametrize("M", [5, 90])
def test_gradients_of_small_and_uneven_scales(M):
    # float16 gradients stay precise whatever the size of the channels' scales
    N, K = 300, 200
    dy = rows(M, M, N, torch.float16)
    w, ws, _ = weights(3, 2, N, K)
    q, xs = ref.quantize(rows(M, M, K))
    # (and of the gradients themselves, where the type can hold them)
    for factor in (2.0 ** -20, 2.0 ** 12):
        s = ws * factor
        s[:, ::7] *= 2.0 ** -3
        want, bound = ref.linear_grad(dy, w[0], s[0])
        dx = q8.linear_per_token_backward(dy.to(DEV), q8.pack_tile_weight(w[0].t().contiguous().to(DEV)),
                                          s[0].contiguous().to(DEV))
        within(dx, want, bound)


@pytest.mark.parametrize("M", [4, 80])
@pytest.mark.parametrize("power", [-100, -60, 60, 90])
def test_gradients_of_far_sizes(M, power):
    # bfloat16 gradients of rows of very different size
    N, K = 140, 200
    dy = (rows(M, M, N) * 2.0 ** (power + torch.arange(M).float()[:, None] / 4)).bfloat16()
    w, ws, b = weights(3, 2, N, K)
    q, xs = ref.quantize(rows(M, M, K))
    want, bound = ref.linear_grad(dy, w[0], ws[0])
    dx = q8.linear_per_token_backward(dy.to(DEV), q8.pack_tile_weight(w[0].t().contiguous().to(DEV)),
                                      ws[0].contiguous().to(DEV))
    within(dx, want, bound)
    g, u = (ref.product(q, xs, w[i], ws[i], b[i]) for i in (0, 1))
    want, bound = ref.gated_grad(dy, g, u, w, ws, "silu", xs, b)
    dx = q8.linear_gated_backward(dy.to(DEV), q.to(DEV), xs.to(DEV), q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV)),
                                  q8.pack_gated_weight_t(w[0].to(DEV), w[1].to(DEV)), ws.to(DEV), b.to(DEV))
    within(dx, want, bound)


def test_channels_past_the_last_take_no_part():
    # rows whose scale is infinite: their own gradients are not finite, the
    # padded channels' zeros stay zeros for the other rows
    M, N, K = 70, 20, 64
    q, xs = ref.quantize(rows(1, M, K))
    dh = rows(2, M, N, torch.bfloat16)
    w, ws, _ = weights(1, 2, N, K)
    packed = q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV))
    packed_t = q8.pack_gated_weight_t(w[0].to(DEV), w[1].to(DEV))
    want = q8.linear_gated_backward(dh.to(DEV), q.to(DEV), xs.to(DEV), packed, packed_t, ws.to(DEV), None)
    xs[3] = float("inf")
    dh[9] = float("nan")
    dx = q8.linear_gated_backward(dh.to(DEV), q.to(DEV), xs.to(DEV), packed, packed_t, ws.to(DEV), None)
    keep = [m for m in range(M) if m not in (3, 9)]
    assert torch.equal(dx[keep], want[keep])
    assert bool(dx[9].isnan().all())


def _loss(x, w, ws, b, act, dh):
    g = (x @ w[0].double().t()) * ws[0].double() + b[0].double()
    u = (x @ w[1].double().t()) * ws[1].double() + b[1].double()
    return (ref.act64(g, act)[0] * u * dh.double()).sum()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_against_differences(act):
    M, N, K = 6, 90, 70
    q, xs = ref.quantize(rows(4, M, K))
    x = q.double() * xs.double()[:, None]
    dh = rows(5, M, N, torch.float16)
    w, ws, b = weights(6, 2, N, K)
    dx = q8.linear_gated_backward(dh.to(DEV), q.to(DEV), xs.to(DEV), q8.pack_gated_weight(w[0].to(DEV), w[1].to(DEV)),
                                  q8.pack_gated_weight_t(w[0].to(DEV), w[1].to(DEV)), ws.to(DEV), b.to(DEV),
                                  activation=act).cpu().double()
    g, u = (ref.product(q, xs, w[i], ws[i], b[i]) for i in (0, 1))
    bound = ref.gated_grad(dh, g, u, w, ws, act, xs, b)[1]
    gen = torch.Generator().manual_seed(7)
    for _ in range(8):
        d = torch.randn(M, K, generator=gen, dtype=torch.float64)
        eps = 1e-5   # the third derivative's part is 1e-10 of the loss's size
        want = (_loss(x + eps * d, w, ws, b, act, dh) - _loss(x - eps * d, w, ws, b, act, dh)) / (2 * eps)
        assert abs(float((dx * d).sum() - want)) <= float((bound * d.abs()).sum()) + 1e-6 * abs(float(want)) + 1e-7


# ---- together ---------------------------------------------------------------

class Block:
    """A feed-forward block of an int8 model."""

    def __init__(self, width, hidden, seed, act="silu"):
        self.w1, self.ws1, self.b1 = weights(seed, 2, hidden, width)
        self.w2, self.ws2, self.b2 = weights(seed + 1, width, hidden)
        self.act = act
        c = lambda t: t.to(DEV)  # noqa: E731
        self.g = q8.pack_gated_weight(c(self.w1[0]), c(self.w1[1]))
        self.gt = q8.pack_gated_weight_t(c(self.w1[0]), c(self.w1[1]))
        self.d = q8.pack_tile_weight(c(self.w2))
        self.dt = q8.pack_tile_weight(c(self.w2.t().contiguous()))
        self.s1, self.c1, self.s2, self.c2 = c(self.ws1), c(self.b1), c(self.ws2), c(self.b2)

    def __call__(self, x):
        h = q8.linear_gated(x, None, self.g, self.s1, self.c1, activation=self.act, packed_t=self.gt)
        return q8.linear_per_token(h, None, self.d, self.s2, self.c2, packed_t=self.dt)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [1, 9, 100])
def test_a_block_and_its_gradient(dtype, M):
    block = Block(160, 333, M)
    x = rows(M, M, 160, dtype).to(DEV).requires_grad_()
    y = block(x)
    dy = rows(M + 1, M, 160, dtype).to(DEV)
    (dx,) = torch.autograd.grad(y, x, dy)
    # the same calls one by one
    with torch.no_grad():
        q, xs = q8.quantize_per_token(x)
        h = q8.linear_gated(q, xs, block.g, block.s1, block.c1, out_dtype=dtype)
        assert torch.equal(y, q8.linear_per_token(h, None, block.d, block.s2, block.c2))
        dh = q8.linear_per_token_backward(dy, block.dt, block.s2)
        assert torch.equal(dx, q8.linear_gated_backward(dh, q, xs, block.g, block.gt, block.s1, block.c1))
    # and the formulas, stage by stage
    qc, xc = q.cpu(), xs.cpu()
    g, u = (ref.product(qc, xc, block.w1[i], block.ws1[i], block.b1[i]) for i in (0, 1))
    within(h, *ref.gated(g, u, "silu", dtype))
    within(dh, *ref.linear_grad(dy.cpu(), block.w2, block.ws2))
    within(dx, *ref.gated_grad(dh.cpu(), g, u, block.w1, block.ws1, "silu", xc, block.b1))


@pytest.mark.parametrize("M,K", [(1, 77), (2, 1003), (7, 130), (30, 333)])
def test_recorded_rows_of_any_length(M, K):
    # the int8 rows and scales that the recorded call keeps are the quantizer's
    N = 60
    x = rows(M, M, K, torch.bfloat16)
    w, ws, b = weights(M, 2, N, K)
    gate, gt = (f(w[0].to(DEV), w[1].to(DEV)) for f in (q8.pack_gated_weight, q8.pack_gated_weight_t))
    leaf = x.to(DEV).requires_grad_()
    h = q8.linear_gated(leaf, None, gate, ws.to(DEV), b.to(DEV), packed_t=gt)
    dh = rows(K, M, N, torch.bfloat16).to(DEV)
    h.backward(dh)
    q, s = q8.quantize_per_token(x.to(DEV))
    assert torch.equal(leaf.grad, q8.linear_gated_backward(dh, q, s, gate, gt, ws.to(DEV), b.to(DEV)))


def test_relu_product_is_recorded():
    w, ws, b = weights(2, 90, 64)
    x = rows(3, 12, 64, torch.bfloat16).to(DEV).requires_grad_()
    pt = q8.pack_tile_weight(w.t().contiguous().to(DEV))
    y = q8.linear_per_token(x, None, q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), b.to(DEV), activation="relu",
                            packed_t=pt)
    dy = rows(4, 12, 90, torch.bfloat16).to(DEV)
    y.backward(dy)
    within(x.grad, *ref.linear_grad(dy.cpu(), w, ws, y.detach().cpu()))
    assert bool((y == 0).any())


def test_float32_rows_get_their_gradient():
    w, ws, b = weights(2, 90, 64)
    x = rows(3, 12, 64).to(DEV).requires_grad_()
    y = q8.linear_per_token(x, None, q8.pack_tile_weight(w.to(DEV)), ws.to(DEV), None, out_dtype=torch.bfloat16,
                            packed_t=q8.pack_tile_weight(w.t().contiguous().to(DEV)))
    y.sum().backward()
    assert x.grad.dtype == torch.float32
    within(x.grad.bfloat16(), *ref.linear_grad(torch.ones(12, 90).bfloat16(), w, ws))


def test_refusals_of_the_binding():
    w, ws, b = weights(2, 2, 90, 64)
    wd, wsd, bd = w.to(DEV), ws.to(DEV), b.to(DEV)
    lin, gate = q8.pack_tile_weight(wd[0]), q8.pack_gated_weight(wd[0], wd[1])
    lt, gt = q8.pack_tile_weight(wd[0].t().contiguous()), q8.pack_gated_weight_t(wd[0], wd[1])
    x = rows(3, 12, 64).to(DEV)
    q, s = q8.quantize_per_token(x)
    s0 = wsd[0].contiguous()
    one = dict(packed=lin, weight_scales=s0, bias=None)
    two = dict(packed=gate, weight_scales=wsd, bias=None)
    refused = [
        (ValueError, lambda: q8.linear_per_token(q, None, **one)),
        (ValueError, lambda: q8.linear_per_token(x, s, **one)),
        (ValueError, lambda: q8.linear_per_token(x[:, :63].contiguous(), None, **one)),
        (ValueError, lambda: q8.linear_per_token(x.t().contiguous().t(), None, **one)),
        (ValueError, lambda: q8.linear_per_token(x.cpu(), None, **one)),
        (TypeError, lambda: q8.linear_per_token(x.double(), None, **one)),
        (TypeError, lambda: q8.linear_per_token(x, None, out_dtype=torch.int8, **one)),
        (TypeError, lambda: q8.linear_per_token(x, None, lin, s0.half(), None)),
        (ValueError, lambda: q8.linear_per_token(x, None, lin, wsd, None)),
        (ValueError, lambda: q8.linear_per_token(q, s[:5], **one)),
        (q8.Q8Error, lambda: q8.linear_per_token(x, None, activation="silu", **one)),
        (q8.Q8Error, lambda: q8.linear_gated(x, None, activation="none", **two)),
        (ValueError, lambda: q8.linear_gated(x, None, gt, wsd, None)),
        (ValueError, lambda: q8.linear_gated(x, None, gate, s0, None)),
        (ValueError, lambda: q8.linear_gated(x.requires_grad_(), None, **two)),
        (TypeError, lambda: q8.linear_gated(x, None, packed_t=gt, **two)),          # float32 outputs
        (ValueError, lambda: q8.linear_gated(x, None, packed_t=gate, out_dtype=torch.float16, **two)),
        (ValueError, lambda: q8.linear_per_token(x.detach(), None, lin, s0.clone().requires_grad_(), None)),
        (TypeError, lambda: q8.linear_per_token_backward(torch.zeros(12, 90, device=DEV), lt, s0)),
        (ValueError, lambda: q8.linear_per_token_backward(torch.zeros(12, 91, device=DEV).half(), lt, s0)),
        (ValueError, lambda: q8.linear_gated_backward(torch.zeros(12, 90, device=DEV).half(), q, s, gate, gate, wsd, None)),
        (ValueError, lambda: q8.linear_gated_backward(torch.zeros(11, 90, device=DEV).half(), q, s, gate, gt, wsd, None)),
        (TypeError, lambda: q8.quantize_per_token(q)),
        (TypeError, lambda: q8.dequantize_per_token(q, s, out_dtype=torch.int8)),
        (ValueError, lambda: q8.dequantize_per_token(q, s[:3])),
        (ValueError, lambda: q8.pack_gated_weight(wd[0], wd[1][:80].contiguous())),
        (ValueError, lambda: q8.linear_per_token(torch.cat([x.detach()] * 3), None, workspace=torch.empty(256, dtype=torch.uint8, device=DEV), **one)),
    ]
    for error, call in refused:
        with pytest.raises(error):
            call()


def test_streams_and_graphs():
    block = Block(256, 300, 1)
    x = rows(5, 24, 256, torch.bfloat16).to(DEV)
    dy = rows(6, 24, 256, torch.bfloat16).to(DEV)

    def step():
        q, xs = q8.quantize_per_token(x)
        h = q8.linear_gated(q, xs, block.g, block.s1, block.c1)
        y = q8.linear_per_token(h, None, block.d, block.s2, block.c2)
        dh = q8.linear_per_token_backward(dy, block.dt, block.s2)
        return h, y, dh, q8.linear_gated_backward(dh, q, xs, block.g, block.gt, block.s1, block.c1)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    other = rows(7, 24, 256, torch.bfloat16).to(DEV)
    x.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, step()))
