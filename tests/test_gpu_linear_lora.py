"""Low-rank adapters beside a shared int8 projection, against the formula in
64 bits.

Bound of a float output's error, from the arithmetic: the adapter-free part is
a chain of four f32 roundings of |acc| s_in ws + |b|; the sum over k runs in f32
(any order, each step 2^-23 relative at most, the tensor core's included), so h
is within (K + 4) 2^-23 of s sum |x A|; h's two tf32 terms leave 2^-21 of |h|;
the sum over ranks adds (2 r + 2) 2^-23; and the output type's rounding adds
u |v|.  Rows without an adapter are compared bit for bit: their value is the
plain linear's.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
DEV = torch.device("cuda:0")
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert q8.device_error(clear=True) == 0


def T(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Problem:
    def __init__(self, seed, M, N, K, L, r, dtype=torch.bfloat16, zp=0, bias=True, ids="random",
                 bare=0.0):
        rng = np.random.default_rng(seed)
        self.M, self.N, self.K, self.L, self.r, self.zp, self.dtype = M, N, K, L, r, zp, dtype
        self.s_in = 0.02
        self.x = np.clip(np.rint(rng.normal(0, 40, (M, K)) + zp), -128, 127).astype(np.int8)
        self.w = rng.integers(-127, 128, (N, K)).astype(np.int8)
        self.ws = (rng.uniform(0.0005, 0.002, N) * np.sqrt(64.0 / K)).astype(np.float32)
        self.b = rng.normal(0, 0.3, N).astype(np.float32) if bias else None
        g = torch.Generator().manual_seed(seed)
        self.A = (torch.randn((L, r, K), generator=g) / np.sqrt(K)).to(dtype)
        self.B = (0.5 * torch.randn((L, N, r), generator=g) / np.sqrt(r)).to(dtype)
        self.s = torch.from_numpy(rng.uniform(0.5, 2.0, L).astype(np.float32))
        a = rng.integers(0, L, M)
        if ids == "runs":
            a = np.sort(a)
        elif ids == "one":
            a = np.full(M, L - 1)
        if bare:
            gone = rng.random(M) < bare
            a[gone] = rng.choice([-1, L, 2 ** 31 - 1, -2 ** 31], size=int(gone.sum()))
        self.a = a.astype(np.int64).astype(np.int32)

    def run(self, out_dtype=torch.float32, act="none", s_out=0.05, z_out=3, **kw):
        packed = q8.pack_tile_weight(T(self.w))
        lora = q8.pack_lora(self.A.to(DEV), self.B.to(DEV), self.s.to(DEV))
        return q8.linear_lora(T(self.x), self.s_in, self.zp, packed, T(self.ws), T(self.b), lora,
                              T(self.a), s_out, z_out, activation=act, out_dtype=out_dtype, **kw)

    def exact(self):
        """(v, bound of |f32 v - v|), 64 bits, before the activation."""
        x = self.x.astype(np.float64) - self.zp
        acc = x @ self.w.astype(np.float64).T
        base = acc * np.float64(np.float32(self.s_in)) * self.ws
        b = np.zeros(self.N) if self.b is None else self.b.astype(np.float64)
        v = base + b
        bound = 2.0 ** -22 * (np.abs(base) + np.abs(b))
        e = 2.0 ** -23
        for l in range(self.L):
            m = self.a == l
            if not m.any():
                continue
            A, B = self.A[l].double().numpy(), self.B[l].double().numpy()
            s = self.s_in * float(self.s[l])
            d = s * (x[m] @ A.T) @ B.T
            size = s * (np.abs(x[m]) @ np.abs(A).T) @ np.abs(B).T
            v[m] += d
            bound[m] += (self.K + 2 * self.r + 16) * e * size + e * np.abs(v[m])
        return v, bound

    def plain(self):
        """The f32 value of rows without an adapter, one rounding per step."""
        acc = (self.x.astype(np.float64) - self.zp) @ self.w.astype(np.float64).T
        v = np.rint(acc).astype(np.int32).astype(np.float32) * np.float32(self.s_in) * self.ws
        return v + (self.b if self.b is not None else np.float32(0)) + np.float32(0)


def _check(p, out_dtype=torch.float32, act="none", **kw):
    got = p.run(out_dtype, act, **kw)
    v, bound = p.exact()
    if act == "relu":
        v = np.maximum(v, 0)
    if out_dtype == torch.int8:
        s_out, z_out = 0.05, 3
        u = v / s_out
        q = got.cpu().numpy().astype(np.float64)
        lo = np.clip(np.rint(u - bound / s_out - 1e-4) + z_out, -128, 127)
        hi = np.clip(np.rint(u + bound / s_out + 1e-4) + z_out, -128, 127)
        assert np.all((q >= lo) & (q <= hi))
    else:
        u = UNIT[out_dtype]
        tiny = 2.0 ** -25 if out_dtype == torch.float16 else 0.0
        err = np.abs(got.double().cpu().numpy() - v)
        limit = bound * (1 + u) + u * np.abs(v) + tiny
        assert np.all(err <= limit), float((err - limit).max())
    bare = (p.a < 0) | (p.a >= p.L)
    if bare.any():
        ref = p.plain()[bare]
        if act == "relu":
            ref = np.maximum(ref, 0)
        if out_dtype == torch.int8:
            if p.N % 4 == 0 and p.K % 4 == 0:
                ref = oracle.linear(p.x[bare], p.s_in, p.zp, p.w, p.ws, p.b, 0.05, 3,
                                    activation=act)
                np.testing.assert_array_equal(got.cpu().numpy()[bare], ref)
        else:
            assert torch.equal(got.cpu()[torch.from_numpy(bare)],
                               torch.from_numpy(ref).to(out_dtype))


# M, N, K, L, r: one row; ranks below, at and beyond 16; ragged N and K; one
# row tile and several; more adapters than rows
SHAPES = [(1, 128, 64, 1, 1), (1, 4096, 1024, 4, 16), (5, 132, 100, 3, 8), (16, 256, 520, 20, 16),
          (33, 4, 4096, 7, 24), (64, 260, 1000, 40, 16), (190, 384, 256, 5, 64),
          (193, 128, 192, 6, 16), (500, 516, 320, 9, 32), (1000, 256, 712, 300, 16),
          (70, 65, 33, 2, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,L,r", SHAPES)
def test_matches_the_formula(M, N, K, L, r, dtype):
    _check(Problem(M + N + r, M, N, K, L, r, dtype, zp=-5, bare=0.15))


@pytest.mark.parametrize("out_dtype", [torch.int8, torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [40, 300])
def test_output_types_and_relu(M, out_dtype):
    _check(Problem(M, M, 196, 712, 8, 16, zp=7, bare=0.2), out_dtype)
    _check(Problem(M + 1, M, 196, 712, 8, 16, torch.float16, zp=-128, bias=False, bare=0.2),
           out_dtype, act="relu")


# Many units for each CTA one after the other, so that the two accumulators
# take turns between sums and adapter terms in every order: few rows an
# adapter, many, none, and tiles of both kinds side by side
@pytest.mark.parametrize("M,N,K,L,ids,bare", [
    (20, 40000, 64, 20, "random", 0.3), (48, 36000, 320, 2, "random", 0.0),
    (130, 20000, 192, 1, "one", 0.0), (500, 8192, 128, 60, "random", 0.1),
    (900, 6000, 64, 5, "runs", 0.5), (400, 8192, 704, 3, "random", 0.9)])
def test_many_units_in_a_row(M, N, K, L, ids, bare):
    _check(Problem(M + L, M, N, K, L, 16, torch.float16, zp=3, ids=ids, bare=bare))


@pytest.mark.parametrize("ids", ["runs", "one"])
@pytest.mark.parametrize("M", [20, 150, 450])
def test_runs_of_one_adapter(M, ids):
    _check(Problem(M, M, 128, 640, 4, 32, zp=2, ids=ids))


def test_no_row_has_an_adapter():
    p = Problem(3, 50, 128, 256, 4, 16, zp=1)
    p.a[:] = -1
    _check(p)
    p = Problem(4, 250, 128, 256, 4, 16, zp=1)
    p.a[:] = 4
    _check(p)


def test_no_rows():
    p = Problem(5, 0, 128, 64, 2, 4)
    assert p.run().shape == (0, 128)


@pytest.mark.parametrize("M", [24, 300])
def test_infinities_stay_with_their_adapter(M):
    p = Problem(6, M, 132, 256, 5, 16, zp=1)
    clean = p.run()
    p.B[2, 7, 3] = float("inf")
    p.A[3, 1, 5] = float("nan")
    got = p.run().cpu()
    bad = torch.from_numpy((p.a == 2) | (p.a == 3))
    assert bad.any() and (~bad).any()
    assert torch.equal(got[~bad], clean.cpu()[~bad])
    assert torch.isnan(got[bad]).all()


def test_large_ranges_of_h():
    """f16 adapters whose h passes f16's range, and tiny ones: h is f32."""
    p = Problem(7, 30, 128, 512, 3, 16, torch.float16, ids="runs")
    p.A = (p.A.float() * 2000).half()
    p.B = (p.B.float() * 1e-3).half()
    _check(p)
    p.A = (p.A.float() * 1e-6).half()
    _check(p)


def test_against_differences():
    """v is linear in B: a central difference in B along a direction is the
    product of h with that direction (16 columns of one adapter), within the
    bound of the two values' errors."""
    p = Problem(8, 12, 64, 128, 2, 16, torch.float16, ids="one")
    step = 2.0 ** -3
    D = torch.zeros_like(p.B)
    D[1, :, 5] = 1.0
    B0 = p.B.clone()
    p.B = (B0.float().mul(1024).round().div(1024) + step * D.float()).half()
    up, bu = p.run().double().cpu().numpy(), p.exact()[1]
    p.B = (B0.float().mul(1024).round().div(1024) - step * D.float()).half()
    down, bd = p.run().double().cpu().numpy(), p.exact()[1]
    h = p.s_in * float(p.s[1]) * (p.x.astype(np.float64) - p.zp) @ p.A[1, 5].double().numpy()
    num = (up - down) / (2 * step)
    assert np.all(np.abs(num - h[:, None]) <= (bu + bd) / (2 * step))


def test_same_bits_every_time_and_workspace_reuse():
    ps = [Problem(20 + i, *s) for i, s in enumerate([(64, 512, 1024, 16, 16), (3, 256, 4096, 8, 64),
                                                    (600, 384, 512, 8, 32)])]
    made = [(q8.pack_tile_weight(T(p.w)),
             q8.pack_lora(p.A.to(DEV), p.B.to(DEV), p.s.to(DEV)), T(p.x), T(p.ws), T(p.b), T(p.a))
            for p in ps]
    size = max(q8.lib().q8_linear_lora_workspace_bytes(p.M, p.K, p.L, p.r) for p in ps)
    space = torch.empty(size, dtype=torch.uint8, device=DEV)
    first = [p.run() for p in ps]
    outs = []
    for _ in range(8):
        for p, (w, l, x, ws, b, a) in zip(ps, made):
            outs.append(q8.linear_lora(x, p.s_in, p.zp, w, ws, b, l, a, 0.05, 3,
                                       out_dtype=torch.float32, workspace=space))
    for i, got in enumerate(outs):
        assert torch.equal(got, first[i % 3])


def test_other_stream_and_graph():
    p = Problem(30, 20, 256, 512, 6, 16)
    ref = p.run()
    packed = q8.pack_tile_weight(T(p.w))
    lora = q8.pack_lora(p.A.to(DEV), p.B.to(DEV), p.s.to(DEV))
    args = (T(p.x), p.s_in, p.zp, packed, T(p.ws), T(p.b), lora, T(p.a), 0.05, 3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = q8.linear_lora(*args, out_dtype=torch.float32)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q8.linear_lora(*args, out_dtype=torch.float32)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


def test_binding_refusals():
    p = Problem(31, 8, 128, 64, 2, 4)
    packed = q8.pack_tile_weight(T(p.w))
    lora = q8.pack_lora(p.A.to(DEV), p.B.to(DEV), p.s.to(DEV))
    ok = dict(x=T(p.x), packed=packed, ws=T(p.ws), b=T(p.b), lora=lora, a=T(p.a))

    def call(**kw):
        c = dict(ok, **{k: v for k, v in kw.items() if k in ok})
        return q8.linear_lora(c["x"], 0.02, 0, c["packed"], c["ws"], c["b"], c["lora"], c["a"], 0.1,
                              0, **{k: v for k, v in kw.items() if k not in ok})
    call()
    two = q8.pack_tile_weight(torch.zeros((2, 128, 64), dtype=torch.int8, device=DEV))
    for bad in (dict(x=T(p.x)[:, :32].contiguous()), dict(a=T(p.a)[:4]), dict(ws=T(p.ws)[:64]),
                dict(packed=two), dict(b=T(p.b)[:3]),
                dict(packed=q8.pack_tile_weight(T(p.w)[:64].contiguous()))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(a=T(p.a).long()), dict(x=T(p.x).float()), dict(out_dtype=torch.int32)):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(q8.Q8Error):
        call(activation="silu")
    A, B, s = p.A.to(DEV), p.B.to(DEV), p.s.to(DEV)
    with pytest.raises(TypeError):
        q8.pack_lora(A.float(), B.float(), s)
    with pytest.raises(TypeError):
        q8.pack_lora(A, B.half(), s)
    with pytest.raises(ValueError):
        q8.pack_lora(A, B[:, :, :2].contiguous(), s)
    with pytest.raises(ValueError):
        q8.pack_lora(A, B, s[:1])
    with pytest.raises(q8.Q8Error):
        q8.pack_lora(torch.zeros((1, 257, 8), dtype=torch.float16, device=DEV),
                     torch.zeros((1, 8, 257), dtype=torch.float16, device=DEV), s[:1])


@pytest.mark.parametrize("M,L,r", [(1, 3, 16), (20, 20, 16), (40, 2, 24), (300, 100, 16),
                                   (300, 5, 40)])
def test_workspace_contents_do_not_matter(M, L, r):
    p = Problem(M + L, M, 260, 320, L, r, torch.float16, zp=4, bare=0.2)
    n = q8.lib().q8_linear_lora_workspace_bytes(p.M, p.K, p.L, p.r)
    _check(p, workspace=torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV))


def test_a_tile_of_many_adapters():
    """One adapter has most rows, some eighty others one each."""
    p = Problem(11, 700, 132, 192, 90, 16, torch.float16, zp=1)
    p.a[:] = 40
    p.a[np.arange(0, 700, 8)] = np.arange(88)
    _check(p)


@pytest.mark.parametrize("M,L", [(20, 20), (40, 2), (100, 3)])
def test_more_exact_chunks_than_accumulators(M, L):
    _check(Problem(M, M, 132, 12000, L, 16, zp=-100, bare=0.1))


# Clusters of 8 CTAs that share a K of one or two blocks, so that most have
# nothing to multiply and reach the exchange of their sums at once: one row tile
# (rows x blocks of 16 ranks up to the SMs) and rows sorted by adapter, one and
# several passes of 64 ranks.  The same bits every time.
@pytest.mark.parametrize("M,L,r", [(1, 1, 16), (2, 2, 256), (9, 3, 16), (64, 1, 24), (70, 2, 16),
                                   (70, 30, 64), (200, 3, 200), (500, 9, 8)])
@pytest.mark.parametrize("K", [20, 64, 128])
def test_clusters_with_little_to_multiply(M, L, r, K):
    p = Problem(M + K, M, 132, K, L, r, zp=3, bare=0.1)
    _check(p)
    first = p.run()
    packed = q8.pack_tile_weight(T(p.w))
    lora = q8.pack_lora(p.A.to(DEV), p.B.to(DEV), p.s.to(DEV))
    args = (T(p.x), p.s_in, p.zp, packed, T(p.ws), T(p.b), lora, T(p.a), 0.05, 3)
    for got in [q8.linear_lora(*args, out_dtype=torch.float32) for _ in range(50)]:
        assert torch.equal(got, first)


# Rows sorted by adapter, their terms row by row: the workspace holds the ids
# of the call before, all of them adapters.  320 blocks, more than CTAs, so that
# a CTA's first part holds a block's end.
def test_ids_of_the_call_before_do_not_matter():
    p = Problem(40, 300, 8192, 128, 100, 16, zp=2)
    packed = q8.pack_tile_weight(T(p.w))
    lora = q8.pack_lora(p.A.to(DEV), p.B.to(DEV), p.s.to(DEV))
    x, ws, b = T(p.x), T(p.ws), T(p.b)
    rng = np.random.default_rng(41)
    ids = [T(rng.permutation(p.a)) for _ in range(2)] + [T(((p.a + 50) % 100).astype(np.int32))]
    n = q8.lib().q8_linear_lora_workspace_bytes(p.M, p.K, p.L, p.r)
    space = torch.empty(n, dtype=torch.uint8, device=DEV)

    def call(a, space=None):
        return q8.linear_lora(x, p.s_in, p.zp, packed, ws, b, lora, a, 0.05, 3,
                              out_dtype=torch.float32, workspace=space)
    want = []
    for a in ids:
        want.append(call(a, torch.zeros(n, dtype=torch.uint8, device=DEV)))
        torch.cuda.synchronize()
    for _ in range(12):
        got = [call(a, space) for a in ids]
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    p.a = ids[2].cpu().numpy()
    v, bound = p.exact()
    u = UNIT[torch.float32]
    assert np.all(np.abs(got[2].double().cpu().numpy() - v) <= bound * (1 + u) + u * np.abs(v))


# Every product positive, so that an infinite scaling makes every channel of its
# adapter's rows infinite, and no others; ranks that fill no block of 16.
@pytest.mark.parametrize("M", [3, 24, 60, 90, 300])
@pytest.mark.parametrize("r", [5, 16, 41])
def test_infinite_scaling(M, r):
    p = Problem(50, M, 132, 200, 5, r, zp=-128)
    p.a[:2] = 2
    p.x = np.maximum(p.x, -127).astype(np.int8)
    p.A, p.B = p.A.abs(), p.B.abs()
    clean = p.run().cpu()
    for s in (float("inf"), -float("inf")):
        p.s[2] = s
        got = p.run().cpu()
        mine = torch.from_numpy(p.a == 2)
        assert bool((got[mine] == s).all())
        assert torch.equal(got[~mine], clean[~mine])


def test_no_rows_with_a_workspace():
    p = Problem(5, 0, 128, 64, 2, 4)
    space = torch.empty(4096, dtype=torch.uint8, device=DEV)
    assert p.run(workspace=space).shape == (0, 128)
    route = q8.expert_sort(torch.zeros((0, 2), dtype=torch.int32, device=DEV), 3)
    packed = q8.pack_tile_weight(torch.zeros((3, 128, 64), dtype=torch.int8, device=DEV))
    got = q8.linear_experts(torch.zeros((0, 64), dtype=torch.int8, device=DEV), 0.02, 0, packed,
                            torch.ones((3, 128), device=DEV), None, route, 0.1, 0, workspace=space)
    assert got.shape == (0, 128)


# h as it is: one input of 1 against A = 1, so that h is the scaling, and B = 1
# (r 1, w 0).  MMAs take h as two terms, which miss it by its last place at most:
# 2^-23 of the power of two below it.  One row tile, narrow and wide, and sorted
# rows; the largest number stays finite (from 2^127 on bits may be cut off), an
# infinity comes through.
@pytest.mark.parametrize("M,L", [(64, 9), (150, 20), (300, 40), (1500, 200)])
def test_h_keeps_its_bits(M, L):
    p = Problem(M, M, 130, 64, L, 1, bias=False)
    p.s_in = 1.0
    p.x[:], p.w[:] = 0, 0
    p.x[:, 3] = 1
    p.A, p.B = torch.zeros_like(p.A), torch.ones_like(p.B)
    p.A[:, 0, 3] = 1
    rng = np.random.default_rng(M)
    s = (rng.uniform(1, 2, L) * 2.0 ** rng.integers(-20, 20, L)).astype(np.float32)
    s[::2] *= -1
    s[:2] = np.float32(3.4028235e38), np.float32("inf")
    p.s = torch.from_numpy(s)
    p.a[:2] = 0, 1
    got = p.run().cpu().numpy()
    want = np.broadcast_to(s[p.a][:, None], got.shape)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine]) and np.isfinite(got[fine]).all()
    fine &= np.abs(want) < 2.0 ** 127
    place = 2.0 ** (np.floor(np.log2(np.abs(want[fine].astype(np.float64)))) - 23)
    assert (np.abs(got[fine].astype(np.float64) - want[fine]) <= place).all()
