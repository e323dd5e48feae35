"""Host-side guards of the entry points for rows that go through different
weights (no GPU needed: every call is refused, or has nothing to do, before
anything is enqueued)."""
import ctypes

import pytest

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
lib = q8.lib()

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced
ODD = ctypes.c_void_p(0x10002)
F32, F16, BF16, I8 = range(4)


def test_sort_guards():
    f = lib.q8_expert_sort
    assert f(None, 4, 2, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_NULL
    assert f(FAKE, 4, 2, 8, None, FAKE, FAKE, None) == q8.Q8_ERR_NULL
    assert f(FAKE, 4, 2, 8, FAKE, None, FAKE, None) == q8.Q8_ERR_NULL
    assert f(None, 0, 2, 8, None, None, None, None) == q8.Q8_ERR_NULL   # offsets are written
    assert f(FAKE, -1, 2, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert f(FAKE, 4, 0, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert f(FAKE, 4, 2, 0, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert f(FAKE, 4, 2, 1025, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert f(FAKE, 2 ** 30, 2, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE   # T*k > INT32_MAX
    assert f(FAKE, 2 ** 62, 4, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert f(FAKE, 4, 2, 8, ODD, FAKE, FAKE, None) == q8.Q8_ERR_ALIGN


def test_gather_and_dispatch_guards():
    g = lib.q8_expert_gather
    assert g(FAKE, 7, 4, 2, 16, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_ARG
    assert g(None, F32, 4, 2, 16, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_NULL
    assert g(FAKE, F32, 4, 2, 16, 8, None, FAKE, FAKE, None) == q8.Q8_ERR_NULL
    assert g(FAKE, F32, 4, 2, 0, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert g(FAKE, F32, 2 ** 20, 2, 2 ** 50, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert g(ODD, F32, 4, 2, 16, 8, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_ALIGN
    assert g(None, F32, 0, 2, 16, 8, None, None, None, None) == q8.Q8_OK       # nothing to move
    d = lib.q8_expert_dispatch
    assert d(None, I8, 4, 16, FAKE, 2, 8, FAKE, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_NULL
    assert d(FAKE, I8, 4, 16, FAKE, 2, 8, FAKE, FAKE, FAKE, None, None) == q8.Q8_ERR_NULL
    assert d(FAKE, 9, 4, 16, FAKE, 2, 8, FAKE, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_ARG
    assert d(FAKE, F16, 4, 16, FAKE, 2, 2000, FAKE, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    assert d(FAKE, F16, 4, 16, None, 2, 8, FAKE, FAKE, FAKE, FAKE, None) == q8.Q8_ERR_NULL


def test_combine_and_gradient_guards():
    c = lib.q8_expert_combine
    assert c(FAKE, I8, FAKE, 4, 2, 16, FAKE, FAKE, None) == q8.Q8_ERR_UNSUPPORTED
    assert c(FAKE, -1, FAKE, 4, 2, 16, FAKE, FAKE, None) == q8.Q8_ERR_ARG
    assert c(FAKE, F32, None, 4, 2, 16, FAKE, FAKE, None) == q8.Q8_ERR_NULL
    assert c(FAKE, F32, FAKE, 4, 2, 16, FAKE, ODD, None) == q8.Q8_ERR_ALIGN
    assert c(FAKE, BF16, FAKE, 4, 2, -1, FAKE, FAKE, None) == q8.Q8_ERR_SHAPE
    b = lib.q8_expert_gather_backward
    assert b(FAKE, I8, 4, 2, 16, FAKE, FAKE, None) == q8.Q8_ERR_UNSUPPORTED
    assert b(FAKE, F32, 4, 2, 16, None, FAKE, None) == q8.Q8_ERR_NULL
    assert b(ODD, F32, 4, 2, 16, FAKE, FAKE, None) == q8.Q8_ERR_ALIGN
    w = lib.q8_expert_combine_backward
    ok = [FAKE, FAKE, F32, FAKE, 4, 2, 16, 8, FAKE, FAKE, FAKE, FAKE, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return w(*a)
    for i in (0, 1, 3, 8, 9, 10, 11):
        assert call(**{f"a{i}": None}) == q8.Q8_ERR_NULL
        assert call(**{f"a{i}": ODD}) == q8.Q8_ERR_ALIGN
    assert call(a2=I8) == q8.Q8_ERR_UNSUPPORTED
    assert call(a7=0) == q8.Q8_ERR_SHAPE


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    ids = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        q8.expert_sort(ids, 4)
    with pytest.raises(ValueError, match="CUDA"):
        q8.expert_dispatch(torch.zeros(2, 8), ids, 4)


def test_tile_pack_guards():
    size = lib.q8_tile_packed_weight_bytes
    assert size(1, 128, 64) == 8192 + 256
    assert size(3, 129, 65) == 3 * 2 * 2 * 8192 + 256
    assert size(0, 128, 64) == size(1, 0, 64) == size(1, 128, 0) == size(1025, 1, 1) == 0
    assert size(1024, 2 ** 30, 2 ** 30) == 0
    p = lib.q8_tile_pack_weight
    assert p(None, 1, 128, 64, FAKE, 1 << 20, None) == q8.Q8_ERR_NULL
    assert p(FAKE, 1, 128, 64, None, 1 << 20, None) == q8.Q8_ERR_NULL
    assert p(FAKE, 0, 128, 64, FAKE, 1 << 20, None) == q8.Q8_ERR_SHAPE
    assert p(FAKE, 1, 128, 64, FAKE, 8192, None) == q8.Q8_ERR_WORKSPACE
    assert p(FAKE, 1, 128, 64, ctypes.c_void_p(0x10010), 1 << 20, None) == q8.Q8_ERR_ALIGN


def test_linear_experts_guards():
    f = lib.q8_linear_experts
    need = lib.q8_linear_experts_workspace_bytes(8, 64, 4)
    assert need > 0 and need % 256 == 0
    assert lib.q8_linear_experts_workspace_bytes(0, 64, 4) == 0
    names = ["x", "sorted", "T", "k", "K", "s_in", "zp", "w", "E", "N", "ws", "b", "order",
             "offsets", "s_out", "ozp", "act", "dt", "out", "space", "bytes", "stream"]
    ok = dict(zip(names, [FAKE, 0, 4, 2, 64, 0.02, 0, FAKE, 4, 32, FAKE, None, FAKE, FAKE, 0.1, 0,
                          b"none", I8, FAKE, FAKE, need, None]))

    def call(**kw):
        return f(*dict(ok, **kw).values())
    for n in ("x", "w", "ws", "order", "offsets", "out", "act"):
        assert call(**{n: None}) == q8.Q8_ERR_NULL, n
    for n in ("T", "k", "K", "E", "N"):
        assert call(**{n: -1}) == q8.Q8_ERR_SHAPE, n
    assert call(E=1025) == q8.Q8_ERR_SHAPE
    assert call(act=b"gelu") == q8.Q8_ERR_UNSUPPORTED
    assert call(dt=4) == q8.Q8_ERR_ARG
    assert call(s_in=0.0) == call(s_out=float("nan")) == q8.Q8_ERR_ARG
    assert call(zp=128) == call(ozp=-129) == q8.Q8_ERR_ARG
    assert call(bytes=need - 1) == call(space=None) == q8.Q8_ERR_WORKSPACE
    for n in ("w", "space"):
        assert call(**{n: ctypes.c_void_p(0x10010)}) == q8.Q8_ERR_ALIGN, n
    assert call(ws=ODD) == call(order=ODD) == q8.Q8_ERR_ALIGN
    assert call(out=ctypes.c_void_p(0x10001), dt=BF16) == q8.Q8_ERR_ALIGN
    assert call(T=0, x=None, out=None) == q8.Q8_OK
    # the k-blocks of all units have to fit 32 bits
    assert call(T=2 ** 22, k=8, N=2 ** 16, K=2 ** 16, bytes=2 ** 62) == q8.Q8_ERR_SHAPE


def test_lora_pack_guards():
    size = lib.q8_lora_packed_bytes
    # B tiles of 4 KB, A rows of 64-padded K, scaling
    assert size(2, 128, 64, 16) == 2 * 4096 + 2 * 16 * 64 * 2 + 256
    assert size(0, 128, 64, 16) == size(1025, 128, 64, 16) == size(1, 128, 64, 257) == 0
    p = lib.q8_lora_pack
    big = 1 << 20
    assert p(None, FAKE, FAKE, F16, 2, 16, 128, 64, FAKE, big, None) == q8.Q8_ERR_NULL
    assert p(FAKE, FAKE, None, F16, 2, 16, 128, 64, FAKE, big, None) == q8.Q8_ERR_NULL
    assert p(FAKE, FAKE, FAKE, F32, 2, 16, 128, 64, FAKE, big, None) == q8.Q8_ERR_UNSUPPORTED
    assert p(FAKE, FAKE, FAKE, 5, 2, 16, 128, 64, FAKE, big, None) == q8.Q8_ERR_ARG
    assert p(FAKE, FAKE, FAKE, BF16, 2, 0, 128, 64, FAKE, big, None) == q8.Q8_ERR_SHAPE
    assert p(FAKE, FAKE, FAKE, BF16, 2, 16, 128, 64, FAKE, 100, None) == q8.Q8_ERR_WORKSPACE
    assert p(ctypes.c_void_p(0x10001), FAKE, FAKE, BF16, 2, 16, 128, 64, FAKE, big,
             None) == q8.Q8_ERR_ALIGN


def test_linear_lora_guards():
    f = lib.q8_linear_lora
    need = lib.q8_linear_lora_workspace_bytes(8, 64, 4, 16)
    assert need > 0 and need % 256 == 0
    assert lib.q8_linear_lora_workspace_bytes(8, 64, 0, 16) == 0
    names = ["x", "M", "K", "s_in", "zp", "w", "N", "ws", "b", "lora", "ldt", "L", "r", "ids",
             "s_out", "ozp", "act", "dt", "out", "space", "bytes", "stream"]
    ok = dict(zip(names, [FAKE, 8, 64, 0.02, 0, FAKE, 32, FAKE, None, FAKE, BF16, 4, 16, FAKE, 0.1,
                          0, b"none", I8, FAKE, FAKE, need, None]))

    def call(**kw):
        return f(*dict(ok, **kw).values())
    for n in ("x", "w", "ws", "lora", "ids", "out", "act"):
        assert call(**{n: None}) == q8.Q8_ERR_NULL, n
    for n in ("M", "K", "N", "L", "r"):
        assert call(**{n: -1}) == q8.Q8_ERR_SHAPE, n
    assert call(r=257) == call(L=1025) == q8.Q8_ERR_SHAPE
    assert call(ldt=F32) == q8.Q8_ERR_UNSUPPORTED
    assert call(act=b"tanh") == q8.Q8_ERR_UNSUPPORTED
    assert call(dt=-1) == q8.Q8_ERR_ARG
    assert call(s_in=-1.0) == call(ozp=200) == q8.Q8_ERR_ARG
    assert call(bytes=need - 1) == call(space=None) == q8.Q8_ERR_WORKSPACE
    for n in ("w", "lora", "space"):
        assert call(**{n: ctypes.c_void_p(0x10010)}) == q8.Q8_ERR_ALIGN, n
    assert call(ids=ODD) == call(out=ODD, dt=F32) == q8.Q8_ERR_ALIGN
    assert call(M=0, x=None, ids=None) == q8.Q8_OK


def test_binding_remembers_workspace_sizes_by_device(monkeypatch):
    """They depend on the device's SMs: a size found on one device is not another's."""
    torch = pytest.importorskip("torch")
    from int8_quantized_q8ta_gb300 import rows
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    class Lib:
        def q8_linear_experts_workspace_bytes(self, R, K, E):
            return 1000 * (current[0] + 1) + R

        def q8_linear_lora_workspace_bytes(self, M, K, L, r):
            return 5000 * (current[0] + 1) + M

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(rows, "_lib", Lib())
    for sizes in (rows._experts_space, rows._lora_space):
        sizes.cache_clear()
    try:
        for _ in range(2):
            for device in (0, 1):
                assert rows._experts_space(7, 64, 4, device) == 1000 * (device + 1) + 7
                assert rows._lora_space(9, 64, 4, 16, device) == 5000 * (device + 1) + 9
    finally:
        for sizes in (rows._experts_space, rows._lora_space):
            sizes.cache_clear()
