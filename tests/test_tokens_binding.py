"""The binding of the calls for rows with a scale for each token (tokens.py),
without a GPU: tensors that stand in for CUDA ones, and a library that notes
what it is asked."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
from int8_quantized_q8ta_gb300 import rows, tokens  # noqa: E402

DEVICE = 3   # where the stand-ins say they are


class OnDevice(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return DEVICE


def stand_in(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


class Library:
    """Answers every query with 4096 bytes and every call with 0, and notes the
    device that was current."""

    def __init__(self, current):
        self.current, self.seen = current, []

    def __getattr__(self, name):
        def f(*args):
            self.seen.append((name, self.current[-1]))
            return 4096 if name.endswith("_bytes") else 0
        return f


@pytest.fixture
def library(monkeypatch):
    current = [0]

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        try:
            yield
        finally:
            current.pop()
    lib = Library(current)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).as_subclass(OnDevice))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    for module in (rows, tokens):
        monkeypatch.setattr(module, "_lib", lib)
        monkeypatch.setattr(module, "_stream", lambda t: 0)
    tokens._bytes.cache_clear()
    yield lib
    tokens._bytes.cache_clear()


def test_calls_run_on_the_device_of_their_rows(library):
    M, N, K = 40, 32, 64
    x, q, s = stand_in(M, K, dtype=torch.float16), stand_in(M, K, dtype=torch.int8), stand_in(M)
    w, ws, ws2 = stand_in(N, K, dtype=torch.int8), stand_in(N), stand_in(2, N)
    dy = stand_in(M, N, dtype=torch.float16)
    data = stand_in(8, dtype=torch.uint8)
    lin, lin_t = q8.PackedTileWeight(data, 1, N, K), q8.PackedTileWeight(data, 1, K, N)
    gate, gate_t = q8.PackedGatedWeight(data, N, K, False), q8.PackedGatedWeight(data, N, K, True)
    calls = {
        "q8_quantize_per_token": lambda: q8.quantize_per_token(x),
        "q8_dequantize_per_token": lambda: q8.dequantize_per_token(q, s),
        "q8_linear_per_token": lambda: q8.linear_per_token(q, s, lin, ws, None),
        "q8_linear_per_token_backward": lambda: q8.linear_per_token_backward(dy, lin_t, ws),
        "q8_linear_gated": lambda: q8.linear_gated(x, None, gate, ws2, None),
        "q8_linear_gated_backward": lambda: q8.linear_gated_backward(dy, q, s, gate, gate_t, ws2, None),
        "q8_gated_pack_weight": lambda: q8.pack_gated_weight(w, w),
        "q8_tile_pack_weight": lambda: q8.pack_tile_weight(w),
    }
    for name, call in calls.items():
        library.seen.clear()
        call()
        ran = [device for n, device in library.seen if n == name]
        assert ran == [DEVICE], name
        assert library.current == [0]


# ---- without the C++ module ----------------------------------------------------

def test_calls_go_their_longer_way_without_the_module(monkeypatch, library):
    import sys
    monkeypatch.setitem(sys.modules, "int8_quantized_q8ta_gb300._torch_calls", None)   # cannot be imported
    monkeypatch.delattr(q8, "_torch_calls", raising=False)
    monkeypatch.setattr(tokens, "_calls", tokens._Calls())
    x = stand_in(4, 64)
    with pytest.warns(RuntimeWarning, match="_torch_calls.so"):
        q, s = q8.quantize_per_token(x)
    assert q.shape == (4, 64) and s.shape == (4,)
    assert [n for n, _ in library.seen] == ["q8_quantize_per_token"]
    q8.dequantize_per_token(q, s)
    assert [n for n, _ in library.seen] == ["q8_quantize_per_token", "q8_dequantize_per_token"]


def test_the_module_is_rebuilt_for_another_torch(monkeypatch):
    from int8_quantized_q8ta_gb300 import _build
    if not _build.up_to_date():
        pytest.skip("not built here")
    monkeypatch.setattr(_build, "_torch_key", lambda: "another torch")
    assert not _build.up_to_date()
