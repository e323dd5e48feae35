"""The experts' int8 products against the oracle's linear, expert by expert.

int8 outputs are compared byte for byte: the accumulator is exact and the
epilogue is the oracle's sequence of f32 steps.  Float outputs are the same f32
value v before the requantization, rounded once: v is rebuilt from the exact
accumulator with numpy float32 in the same order, and compared bit for bit.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
DEV = torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert q8.device_error(clear=True) == 0


def T(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _problem(seed, T_, k, E, N, K, drop=0.0, bias=True, lo=-127, hi=127, skew=False):
    rng = np.random.default_rng(seed)
    if skew:
        ids = np.minimum(rng.geometric(0.4, (T_, k)) - 1, E - 1)
    else:
        ids = rng.integers(0, E, (T_, k))
    ids = ids.astype(np.int32)
    if drop:
        ids[rng.random((T_, k)) < drop] = -1
    x = rng.integers(-128, 128, (T_, K)).astype(np.int8)
    w = rng.integers(lo, hi + 1, (E, N, K)).astype(np.int8)
    ws = rng.uniform(0.001, 0.005, (E, N)).astype(np.float32)
    b = rng.normal(0, 0.3, (E, N)).astype(np.float32) if bias else None
    return ids, x, w, ws, b


def _accumulators(ids, x, zp, w, k):
    """Sorted rows' exact accumulators, their experts, and the kept count."""
    E, N, _ = w.shape
    flat = ids.reshape(-1)
    rows = [f for e in range(E) for f in np.nonzero(flat == e)[0]]
    acc = np.zeros((flat.size, N), np.int64)
    who = np.zeros(flat.size, np.int64)
    at = 0
    for e in range(E):
        mine = np.nonzero(flat == e)[0]
        if mine.size:
            xs = x[mine // k].astype(np.float64) - zp
            acc[at:at + mine.size] = np.rint(xs @ w[e].astype(np.float64).T).astype(np.int64)
            who[at:at + mine.size] = e
            at += mine.size
    return acc, who, len(rows)


def _value(acc, who, kept, s_in, ws, b, relu):
    """The f32 value before the requantization, one rounding per step."""
    wrapped = ((acc + 2 ** 31) % 2 ** 32 - 2 ** 31).astype(np.int32)
    v = wrapped.astype(np.float32) * np.float32(s_in)
    v = v * ws[who]
    v = v + (b[who] if b is not None else np.float32(0))
    v = v + np.float32(0)
    if relu:
        v = np.maximum(v, np.float32(0))
    v[kept:] = 0
    return v


def _check(seed, T_, k, E, N, K, zp=0, relu=False, out_scale=0.7, ozp=1, x_sorted=False,
           dtypes=(torch.int8, torch.float32, torch.bfloat16, torch.float16), **kw):
    s_in = 0.02 * np.sqrt(64.0 / K)
    ids, x, w, ws, b = _problem(seed, T_, k, E, N, K, **kw)
    route = q8.expert_sort(T(ids), E)
    packed = q8.pack_tile_weight(T(w))
    acc, who, kept = _accumulators(ids, x, zp, w, k)
    act = "relu" if relu else "none"
    xt = T(x)
    if x_sorted:
        xt = q8.expert_gather(xt, route)
    v = _value(acc, who, kept, s_in, ws, b, relu)
    for dt in dtypes:
        out = torch.full((T_ * k, N), 9, dtype=dt, device=DEV)
        got = q8.linear_experts(xt, s_in, zp, packed, T(ws), T(b), route, out_scale, ozp,
                                activation=act, x_sorted=x_sorted, out_dtype=dt, out=out)
        if dt == torch.int8:
            ref = np.full((T_ * k, N), ozp, np.int8)
            for e in np.unique(who[:kept]):
                m = np.nonzero(who[:kept] == e)[0]
                token = route.order.cpu().numpy()[m] // k
                if (w.shape[1] % 4 == 0) and (K % 4 == 0):
                    ref[m] = oracle.linear(np.ascontiguousarray(x[token]), s_in, zp, w[e], ws[e],
                                           None if b is None else b[e], out_scale, ozp,
                                           activation=act)
                else:
                    u = v[m] * np.float32(1.0 / out_scale)
                    ref[m] = np.clip(np.rint(u) + np.float32(ozp), -128, 127).astype(np.int8)
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        else:
            ref = torch.from_numpy(v).to(dt)
            assert torch.equal(got.cpu(), ref), (dt, (got.cpu() != ref).sum())


# T, k, E, N, K: one row; rows of a tile's every size class; N and K that are
# not multiples of the tile; K below one block; groups of several tiles
SHAPES = [(1, 1, 1, 4, 4), (1, 8, 16, 128, 64), (5, 2, 4, 132, 100), (16, 8, 64, 256, 512),
          (40, 3, 5, 36, 1000), (64, 4, 3, 260, 68), (300, 2, 4, 384, 320), (200, 4, 2, 128, 1536),
          (700, 1, 3, 516, 2052), (33, 6, 700, 64, 192), (3, 2, 9, 4, 8192)]


@pytest.mark.parametrize("T_,k,E,N,K", SHAPES)
def test_matches_the_oracle(T_, k, E, N, K):
    _check(T_ + N, T_, k, E, N, K, zp=-7)


@pytest.mark.parametrize("zp", [-128, -3, 0, 5, 127])
@pytest.mark.parametrize("relu", [False, True])
def test_zero_points_and_relu(zp, relu):
    _check(zp + 200, 60, 3, 7, 196, 712, zp=zp, relu=relu, drop=0.2, ozp=-9, bias=not relu,
           dtypes=(torch.int8, torch.float32))


@pytest.mark.parametrize("N,K", [(1, 1), (3, 7), (129, 65), (127, 63), (255, 130)])
def test_any_n_and_k(N, K):
    _check(N * K, 29, 2, 3, N, K, zp=11, dtypes=(torch.int8, torch.float32))


def test_sorted_input():
    _check(5, 50, 4, 6, 256, 384, zp=3, x_sorted=True, drop=0.15)


def test_experts_without_rows_and_one_with_most():
    _check(6, 500, 2, 12, 128, 256, zp=1, skew=True, dtypes=(torch.int8, torch.float32))


def test_every_slot_dropped():
    ids, x, w, ws, b = _problem(7, 6, 2, 3, 64, 64)
    ids[:] = -1
    route = q8.expert_sort(T(ids), 3)
    packed = q8.pack_tile_weight(T(w))
    out = torch.full((12, 64), 9, dtype=torch.int8, device=DEV)
    q8.linear_experts(T(x), 0.02, 0, packed, T(ws), T(b), route, 0.1, -5, out=out)
    assert bool((out == -5).all())
    f = q8.linear_experts(T(x), 0.02, 0, packed, T(ws), T(b), route, 0.1, -5,
                          out_dtype=torch.float16)
    assert bool((f == 0).all())


def test_exact_at_the_chunk_bound():
    """|x - zp| = 255 against |w| = 128 along a long K: f32 partial sums would
    pass 2^24 after 8 blocks of 64, so chunks have to be cut there."""
    E, N, K, T_ = 2, 130, 4096, 40
    rng = np.random.default_rng(3)
    ids = rng.integers(0, E, (T_, 1)).astype(np.int32)
    x = np.full((T_, K), -128, np.int8)
    x[:, ::7] = 127 - rng.integers(0, 3, x[:, ::7].shape)
    w = np.full((E, N, K), -128, np.int8)
    w[1, 1::2] = rng.integers(-128, 128, w[1, 1::2].shape)
    ws = np.full((E, N), 1.0, np.float32)
    route = q8.expert_sort(T(ids), E)
    packed = q8.pack_tile_weight(T(w))
    acc, who, kept = _accumulators(ids, x, 127, w, 1)
    got = q8.linear_experts(T(x), 1.0, 127, packed, T(ws), None, route, 1.0, 0,
                            out_dtype=torch.float32)
    np.testing.assert_array_equal(got.cpu().numpy(), acc.astype(np.float32))


def test_workspace_reuse_and_back_to_back_calls():
    """Calls of different sizes on one workspace, with no wait between them."""
    probs = []
    for i, (T_, k, E, N, K) in enumerate([(64, 4, 8, 256, 1024), (3, 2, 8, 128, 4096),
                                          (400, 2, 4, 384, 512)]):
        ids, x, w, ws, b = _problem(30 + i, T_, k, E, N, K)
        acc, who, kept = _accumulators(ids, x, 2, w, k)
        probs.append((q8.expert_sort(T(ids), E), T(x), q8.pack_tile_weight(T(w)), T(ws), T(b),
                      _value(acc, who, kept, 0.01, ws, b, False), T_ * k, K, E))
    size = max(q8.lib().q8_linear_experts_workspace_bytes(p[6], p[7], p[8]) for p in probs)
    space = torch.empty(size, dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(6):
        for r, x, pk, ws, b, ref, *_ in probs:
            outs.append((q8.linear_experts(x, 0.01, 2, pk, ws, b, r, 1.0, 0,
                                           out_dtype=torch.float32, workspace=space), ref))
    for got, ref in outs:
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


def test_other_stream_and_graph():
    ids, x, w, ws, b = _problem(50, 24, 2, 4, 256, 512)
    route = q8.expert_sort(T(ids), 4)
    packed = q8.pack_tile_weight(T(w))
    args = (T(x), 0.01, 2, packed, T(ws), T(b), route, 1.0, 0)
    ref = q8.linear_experts(*args, out_dtype=torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = q8.linear_experts(*args, out_dtype=torch.float32)
    side.synchronize()
    assert torch.equal(got, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q8.linear_experts(*args, out_dtype=torch.float32)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, ref)


def test_offsets_from_elsewhere_stay_inside():
    """Offsets that a program wrote itself are clamped to the rows there are."""
    ids, x, w, ws, b = _problem(51, 16, 1, 2, 128, 128)
    route = q8.expert_sort(T(ids), 2)
    packed = q8.pack_tile_weight(T(w))
    good = q8.linear_experts(T(x), 0.02, 0, packed, T(ws), T(b), route, 1.0, 0,
                             out_dtype=torch.float32)
    n0 = int(route.offsets[1])
    wide = q8.ExpertRoute(route.order, route.position,
                          torch.tensor([-5, n0, 10 ** 9], dtype=torch.int32, device=DEV))
    got = q8.linear_experts(T(x), 0.02, 0, packed, T(ws), T(b), wide, 1.0, 0,
                            out_dtype=torch.float32)
    assert torch.equal(got, good)


def test_binding_refusals():
    ids, x, w, ws, b = _problem(52, 8, 2, 4, 64, 64)
    route = q8.expert_sort(T(ids), 4)
    packed = q8.pack_tile_weight(T(w))
    ok = dict(x=T(x), ws=T(ws), b=T(b), route=route)

    def call(**kw):
        a = dict(ok, **{k: v for k, v in kw.items() if k in ok})
        more = {k: v for k, v in kw.items() if k not in ok}
        return q8.linear_experts(a["x"], 0.02, 0, packed, a["ws"], a["b"], a["route"], 0.1, 0,
                                 **more)
    call()
    for bad in (dict(x=T(x)[:4]), dict(ws=T(ws)[:, :32].contiguous()), dict(b=T(b)[:2]),
                dict(route=q8.expert_sort(T(ids), 5)), dict(x_sorted=True),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(x=T(x).float()), dict(ws=T(ws).half()), dict(out_dtype=torch.float64)):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(q8.Q8Error):
        call(activation="gelu")
    with pytest.raises(ValueError):
        q8.pack_tile_weight(T(w)[0, 0])


# Output blocks cut between CTAs, and joined: two or more CTAs to each of a few
# blocks; runs that end one block and begin the next, in both forms
@pytest.mark.parametrize("M,N,K", [(8, 1024, 4096), (20, 25600, 3456), (64, 6144, 4100),
                                   (100, 25600, 2688), (150, 2048, 4096)])
def test_blocks_cut_between_ctas(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M)
    x = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand(1, N, generator=g, device=DEV) * 0.004 + 0.001
    route = q8.expert_sort(torch.zeros(M, 1, dtype=torch.int32, device=DEV), 1)
    packed = q8.pack_tile_weight(w)
    acc = torch.cat([(x.double() + 7) @ part.double().T for part in w.split(4096)], 1)
    v = acc.float() * torch.tensor(np.float32(0.01), device=DEV) * ws
    for _ in range(3):   # (joins depend on which CTA comes last, results must not)
        got = q8.linear_experts(x, 0.01, -7, packed, ws, None, route, 1.0, 0,
                                out_dtype=torch.float32)
        assert torch.equal(got, v + 0.0)


# Joined parts are those of this call: problems with other sums in turn on one
# workspace, so that a part read early would be one of the call before.  Units
# shared by several CTAs, and runs that end one unit and begin the next, in both
# forms.
@pytest.mark.parametrize("M,N,K", [(3, 512, 8192), (20, 25600, 4096), (100, 2048, 4096),
                                   (100, 25600, 4096)])
def test_parts_of_the_call_before_do_not_matter(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M + 1)
    x = [torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
         for _ in range(2)]
    w = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    ones = torch.ones(1, N, device=DEV)
    route = q8.expert_sort(torch.zeros(M, 1, dtype=torch.int32, device=DEV), 1)
    packed = q8.pack_tile_weight(w)
    n = q8.lib().q8_linear_experts_workspace_bytes(M, K, 1)
    space = torch.empty(n, dtype=torch.uint8, device=DEV)
    want = [(a.double() @ w.double().T).float() for a in x]
    for _ in range(20):
        got = [q8.linear_experts(a, 1.0, 0, packed, ones, None, route, 1.0, 0,
                                 out_dtype=torch.float32, workspace=space) for a in x]
        for v, ref in zip(got, want):
            assert torch.equal(v, ref)


def test_offsets_that_overlap():
    """Offsets that fall again give groups far more tiles than disjoint ones have
    (512 groups of all 1024 rows: 32768 tiles instead of 1087 at most, whose k-blocks
    pass 32 bits in large problems).  Rows outside the output stay as they
    are, and the next call is right."""
    R, E, N, K = 1024, 1023, 132, 200
    rng = np.random.default_rng(60)
    x = rng.integers(-128, 128, (R, K)).astype(np.int8)
    w = rng.integers(-127, 128, (E, N, K)).astype(np.int8)
    ws = np.full((E, N), 0.01, np.float32)
    route = q8.expert_sort(T(rng.integers(0, E, (R, 1)).astype(np.int32)), E)
    packed = q8.pack_tile_weight(T(w))
    fallen = torch.tensor([0, R] * (E // 2 + 1), dtype=torch.int32, device=DEV)[:E + 1]
    wrong = q8.ExpertRoute(route.order, route.position, fallen.contiguous())
    space = torch.full((R + 64, N), 1e30, device=DEV)
    q8.linear_experts(T(x), 0.02, 3, packed, T(ws), None, wrong, 1.0, 0, out_dtype=torch.float32,
                      out=space[32:-32])
    untouched = space == torch.tensor(1e30, device=DEV)
    assert bool(untouched[:32].all()) and bool(untouched[-32:].all())
    assert not bool(untouched[32:-32].any())
    got = q8.linear_experts(T(x), 0.02, 3, packed, T(ws), None, route, 1.0, 0,
                            out_dtype=torch.float32)
    order = route.order.cpu().numpy()
    who = np.searchsorted(route.offsets.cpu().numpy()[1:], np.arange(R), side="right")
    acc = np.einsum("rk,rnk->rn", x[order].astype(np.float64) - 3, w[who].astype(np.float64))
    v = acc.astype(np.float32) * np.float32(0.02) * ws[who] + np.float32(0)
    np.testing.assert_array_equal(got.cpu().numpy(), v)


FIRST_CALLS = r"""
import sys, threading
sys.path.insert(0, sys.argv[1])
import torch
import int8_quantized_q8ta_gb300 as q8
dev = torch.device("cuda:0")
g = torch.Generator(device=dev).manual_seed(1)
x = torch.randint(-128, 128, (150, 512), generator=g, device=dev, dtype=torch.int8)
w = torch.randint(-127, 128, (384, 512), generator=g, device=dev, dtype=torch.int8)
ones = torch.ones(1, 384, device=dev)
route = q8.expert_sort(torch.zeros(150, 1, dtype=torch.int32, device=dev), 1)
packed = q8.pack_tile_weight(w)
want = (x.double() @ w.double().T).float()
torch.cuda.synchronize()
start, good = threading.Barrier(8), []

def call():
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        out = [q8.linear_experts(x, 1.0, 0, packed, ones, None, route, 1.0, 0,
                                 out_dtype=torch.float32) for _ in range(5)]
        torch.cuda.current_stream().synchronize()
        good.append(all(torch.equal(v, want) for v in out))

threads = [threading.Thread(target=call) for _ in range(8)]
[t.start() for t in threads]
[t.join() for t in threads]
assert good == [True] * 8, good
assert q8.device_error() == 0
"""


def test_first_calls_of_several_threads():
    """A process whose first calls of the wide form come from eight threads."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS, root], capture_output=True, text=True,
                          timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]
