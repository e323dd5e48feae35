"""Host-side guards of the entry points for rows with a scale for each token
(no GPU needed: every call is refused, or has nothing to do, before anything is
enqueued)."""
import ctypes

import pytest

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
lib = q8.lib()

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10080)  # not on 256 bytes
F32, F16, BF16, I8 = range(4)


def caller(f, **ok):
    return lambda **kw: f(*dict(ok, **kw).values())


def test_quantize_and_back_guards():
    q = caller(lib.q8_quantize_per_token, x=FAKE, dt=F32, M=4, K=64, q=FAKE, s=FAKE, stream=None)
    d = caller(lib.q8_dequantize_per_token, q=FAKE, s=FAKE, M=4, K=64, dt=F32, out=FAKE, stream=None)
    for call, names in ((q, ("x", "q", "s")), (d, ("q", "s", "out"))):
        for n in names:
            assert call(**{n: None}) == q8.Q8_ERR_NULL, n
        assert call(dt=4) == call(dt=-1) == q8.Q8_ERR_ARG
        assert call(dt=I8) == q8.Q8_ERR_UNSUPPORTED
        assert call(M=-1) == call(K=0) == call(M=2 ** 31) == call(K=2 ** 31) == q8.Q8_ERR_SHAPE
        assert call(M=0, **{n: None for n in names}) == q8.Q8_OK
        assert call(s=ODD) == q8.Q8_ERR_ALIGN
    assert q(x=ODD) == q(x=ODD, dt=F16) == d(out=ODD) == d(out=ODD, dt=BF16) == q8.Q8_ERR_ALIGN


@pytest.mark.parametrize("gated", [False, True])
def test_product_guards(gated):
    M, K, N = 40, 64, 32
    f = lib.q8_linear_gated if gated else lib.q8_linear_per_token
    query = lib.q8_linear_gated_workspace_bytes if gated else lib.q8_linear_per_token_workspace_bytes
    need = query(M, K, N)
    assert need > 0 and need % 256 == 0
    assert query(1, K, N) == query(0, K, N) == query(M, 0, N) == query(M, K, 0) == 0
    call = caller(f, x=FAKE, dt=BF16, M=M, K=K, q=None, s=None, w=FAKE, N=N, ws=FAKE, b=None,
                  act=b"silu" if gated else b"none", out_dt=BF16, out=FAKE, space=FAKE, bytes=need, stream=None)
    for n in ("x", "w", "ws", "out", "act"):
        assert call(**{n: None}) == q8.Q8_ERR_NULL, n
    assert call(dt=I8) == q8.Q8_ERR_NULL                       # int8 rows come with scales
    for n in ("M", "K", "N"):
        assert call(**{n: -1}) == call(**{n: 2 ** 31}) == q8.Q8_ERR_SHAPE, n
    assert call(K=0) == call(N=0) == call(N=2 ** 24 + 1) == q8.Q8_ERR_SHAPE
    assert call(dt=4) == call(out_dt=-1) == q8.Q8_ERR_ARG
    assert call(out_dt=I8) == q8.Q8_ERR_UNSUPPORTED
    for act in (b"tanh", b"", b"none" if gated else b"silu"):
        assert call(act=act) == q8.Q8_ERR_UNSUPPORTED
    assert call(bytes=need - 1) == call(space=None) == q8.Q8_ERR_WORKSPACE
    for n in ("w", "space"):
        assert call(**{n: HALF}) == q8.Q8_ERR_ALIGN, n
    for n in ("x", "ws", "b", "out", "s"):
        assert call(**{n: ODD}) == q8.Q8_ERR_ALIGN, n
    assert call(M=0, x=None, w=None, ws=None, out=None) == q8.Q8_OK


def test_gradient_guards():
    M, N, K = 40, 32, 64
    need = lib.q8_linear_per_token_backward_workspace_bytes(M, N, K)
    assert need > 0 and need % 256 == 0 and lib.q8_linear_per_token_backward_workspace_bytes(0, N, K) == 0
    one = caller(lib.q8_linear_per_token_backward, dy=FAKE, dt=BF16, M=M, N=N, y=None, w=FAKE, K=K, ws=FAKE, out=FAKE,
                 space=FAKE, bytes=need, stream=None)
    need2 = lib.q8_linear_gated_backward_workspace_bytes(M, K, N)
    assert need2 > 0 and need2 % 256 == 0 and lib.q8_linear_gated_backward_workspace_bytes(M, K, 0) == 0
    two = caller(lib.q8_linear_gated_backward, dy=FAKE, dt=BF16, M=M, N=N, q=FAKE, s=FAKE, K=K, w=FAKE, wt=FAKE, ws=FAKE,
                 b=None, act=b"silu", out=FAKE, space=FAKE, bytes=need2, stream=None)
    for call, need_, names in ((one, need, ("dy", "w", "ws", "out")), (two, need2, ("dy", "q", "s", "w", "wt", "ws", "out"))):
        for n in names:
            assert call(**{n: None}) == q8.Q8_ERR_NULL, n
        assert call(dt=F32) == call(dt=I8) == q8.Q8_ERR_UNSUPPORTED
        assert call(dt=4) == q8.Q8_ERR_ARG
        for n in ("M", "N", "K"):
            assert call(**{n: -1}) == q8.Q8_ERR_SHAPE, n
        assert call(bytes=need_ - 1) == call(space=None) == q8.Q8_ERR_WORKSPACE
        assert call(w=HALF) == call(space=HALF) == call(dy=ODD) == call(out=ODD) == call(ws=ODD) == q8.Q8_ERR_ALIGN
        assert call(M=0, **{n: None for n in names}) == q8.Q8_OK
    assert one(y=ODD) == two(b=ODD) == two(s=ODD) == two(wt=HALF) == q8.Q8_ERR_ALIGN
    assert two(act=b"none") == q8.Q8_ERR_UNSUPPORTED and two(act=None) == q8.Q8_ERR_NULL


def test_gated_pack_guards():
    size = lib.q8_gated_packed_weight_bytes
    assert size(64, 64, 0) == 8192 + 256                       # 128 packed rows
    assert size(65, 65, 0) == 2 * 2 * 8192 + 256
    assert size(64, 128, 1) == 2 * 8192 + 256                  # 128 rows of 128 packed inputs
    assert size(0, 64, 0) == size(64, 0, 0) == size(2 ** 23 + 1, 1, 0) == size(2 ** 23, 2 ** 40, 1) == 0
    call = caller(lib.q8_gated_pack_weight, gate=FAKE, up=FAKE, N=64, K=64, t=0, dst=FAKE, bytes=1 << 20, stream=None)
    for n in ("gate", "up", "dst"):
        assert call(**{n: None}) == q8.Q8_ERR_NULL, n
    assert call(N=0) == call(K=-1) == q8.Q8_ERR_SHAPE
    assert call(bytes=8192) == q8.Q8_ERR_WORKSPACE
    assert call(dst=HALF) == q8.Q8_ERR_ALIGN


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x, q = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8)
    w = torch.zeros(32, 64, dtype=torch.int8)
    for call in (lambda: q8.quantize_per_token(x), lambda: q8.dequantize_per_token(q, torch.ones(2)),
                 lambda: q8.pack_gated_weight(w, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        q8.quantize_per_token([1.0, 2.0])
