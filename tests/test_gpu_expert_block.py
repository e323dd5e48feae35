"""The example block's stages against plain PyTorch in 64 bits.

int8 stages may be one step off where the exact value lies on a rounding
boundary (their f32 steps err by some 2^-22 of it); bf16 ones are rounded once
(2^-8 of the largest value at most, 2^-7 allowed for a boundary and f32's own
error).
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

q8 = pytest.importorskip("int8_quantized_q8ta_gb300")
PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "expert_block.py")


def _example():
    spec = importlib.util.spec_from_file_location("expert_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("tokens,experts,k", [(1, 16, 4), (37, 5, 2), (300, 16, 4)])
def test_block(tokens, experts, k):
    example = _example()
    block = example.ExpertBlock(width=256, hidden=324, experts=experts, k=k, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, 256, generator=g, device="cuda")
    ids = torch.randint(-1, block.L, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    for name, e in example.errors(block, x, ids).items():
        assert e <= (1 if "steps" in name else 2.0 ** -7), (name, e)
    assert q8.device_error() == 0


def test_gradients():
    example = _example()
    block = example.ExpertBlock(width=128, hidden=192)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(50, 128, generator=g, device="cuda")
    y, kept = block.forward(x, torch.zeros(50, dtype=torch.int32, device="cuda"))
    dy = torch.randn(50, 128, generator=g, device="cuda").bfloat16()
    dz, dw, dx = block.backward(dy, kept)
    z = kept["z"].double().requires_grad_()
    w = kept["weights"].double().requires_grad_()
    position = kept["route"].position.long()
    (z[position] * w[:, :, None]).sum(1).backward(dy.double())
    assert (dz.double() - z.grad).abs().max() <= 2.0 ** -8 * z.grad.abs().max()
    # 128 products summed in f32, each within 2^-23 of its size
    size = (dy.double()[:, None, :] * z.detach()[position]).abs().sum(2)
    assert ((dw.double() - w.grad).abs() <= 130 * 2.0 ** -23 * size).all()
    # four bf16 rows added in f32 and rounded once
    want = dz.double()[position].sum(1)
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-30 + 4 * 2.0 ** -23 *
            dz.double()[position].abs().sum(1)).all()
