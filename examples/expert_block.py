"""One int8 block of a mixture model that serves many adapters: a shared
projection with each request's low-rank adapter, a router, the experts' two
products, and the sum back to tokens; then the gradients that train the router.

    python examples/expert_block.py [tokens]

prints the block's time and how far its stages are from plain PyTorch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import int8_quantized_q8ta_gb300 as q8  # noqa: E402


class ExpertBlock:
    """Random weights of the given sizes, packed once."""

    def __init__(self, width=512, hidden=768, experts=16, k=4, adapters=12, rank=16, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def ints(*shape):
            return torch.randint(-127, 128, shape, generator=g, device=device, dtype=torch.int8)

        def real(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device=device) * scale

        self.k, self.E, self.L = k, experts, adapters
        self.w = {"proj": ints(width, width), "up": ints(experts, hidden, width),
                  "down": ints(experts, width, hidden)}
        self.ws = {n: torch.full(w.shape[:-1], 1.0 / (73.0 * w.shape[-1] ** 0.5), device=device)
                   for n, w in self.w.items()}
        self.b = {n: real(*w.shape[:-1], scale=0.1) for n, w in self.w.items()}
        self.A = real(adapters, rank, width, scale=width ** -0.5).bfloat16()
        self.B = real(adapters, width, rank, scale=0.3 * rank ** -0.5).bfloat16()
        self.scaling = torch.full((adapters,), 0.5, device=device)
        self.router = real(experts, width, scale=width ** -0.5)
        self.scale = {"x": 0.03, "proj": 0.03, "up": 0.04}   # int8 steps of the activations
        self.packed = {n: q8.pack_tile_weight(w) for n, w in self.w.items()}
        self.lora = q8.pack_lora(self.A, self.B, self.scaling)

    def route(self, h):
        """Each token's k experts and their weights, from int8 h."""
        logits = (h.float() * self.scale["proj"]) @ self.router.T
        top, ids = logits.topk(self.k, dim=1)
        return ids.int(), torch.softmax(top, dim=1)

    def forward(self, x, adapter_ids):
        """x float32 [T, width], adapter_ids int32 [T] (out of range: none)."""
        s = self.scale
        xq = q8.quantize_per_tensor(x, s["x"], 0)
        h = q8.linear_lora(xq, s["x"], 0, self.packed["proj"], self.ws["proj"], self.b["proj"],
                           self.lora, adapter_ids, s["proj"], 0)
        ids, weights = self.route(h)
        rows, route = q8.expert_dispatch(h, ids, self.E)
        up = q8.linear_experts(rows, s["proj"], 0, self.packed["up"], self.ws["up"], self.b["up"],
                               route, s["up"], 0, activation="relu", x_sorted=True)
        z = q8.linear_experts(up, s["up"], 0, self.packed["down"], self.ws["down"],
                              self.b["down"], route, 1.0, 0, x_sorted=True,
                              out_dtype=torch.bfloat16)
        y = q8.expert_combine(z, weights, route)
        return y, {"xq": xq, "h": h, "ids": ids, "weights": weights, "route": route, "rows": rows,
                   "up": up, "z": z}

    def backward(self, dy, kept):
        """(dz, dweights, dx): the gradients of the experts' outputs and of the
        router's weights, and the gather's gradient taken of dz.  The int8
        products between rows and z have no gradient, so dz stands in for the
        rows' own: dx shows the move back to tokens and is not the block's
        gradient of them."""
        dz, dw = q8.expert_combine_backward(dy, kept["z"], kept["weights"], kept["route"])
        return dz, dw, q8.expert_gather_backward(dz, kept["route"])

    # ---- the same stages in plain PyTorch, each from the block's own inputs ---

    def plain_linear(self, name, x, step, e=None):
        w = self.w[name] if e is None else self.w[name][e]
        ws, b = (self.ws[name], self.b[name]) if e is None else (self.ws[name][e], self.b[name][e])
        return (x.double() @ w.double().T) * step * ws.double() + b.double()

    def plain(self, kept, adapter_ids):
        """(h, up, z, y) in 64 bits, before any quantization or rounding."""
        s, route = self.scale, kept["route"]
        h = self.plain_linear("proj", kept["xq"], s["x"])
        for a in range(self.L):
            m = adapter_ids == a
            xa = kept["xq"][m].double() @ self.A[a].double().T
            h[m] += s["x"] * float(self.scaling[a]) * (xa @ self.B[a].double().T)
        bounds = route.offsets.tolist()
        parts = [(e, slice(bounds[e], bounds[e + 1])) for e in range(self.E)]
        up = torch.cat([self.plain_linear("up", kept["rows"][m], s["proj"], e) for e, m in parts])
        z = torch.cat([self.plain_linear("down", kept["up"][m], s["up"], e) for e, m in parts])
        slots = kept["z"].double()[route.position.long()]
        return h, up.clamp(min=0), z, (slots * kept["weights"].double()[:, :, None]).sum(1)


def errors(block, x, adapter_ids):
    """Largest differences from the plain stages: int8 ones in steps."""
    y, kept = block.forward(x, adapter_ids)
    h, up, z, total = block.plain(kept, adapter_ids)
    s = block.scale

    def steps(q, v, step):
        return float((q.double() - (v / step).round().clamp(-128, 127)).abs().max())

    def relative(got, want):
        return float((got.double() - want).abs().max() / want.abs().max())

    return {"projection (steps)": steps(kept["h"], h, s["proj"]),
            "experts up (steps)": steps(kept["up"], up, s["up"]),
            "experts down (relative)": relative(kept["z"], z),
            "combine (relative)": relative(y, total)}


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 256
    block = ExpertBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, 512, generator=g, device="cuda")
    adapter_ids = torch.randint(-1, block.L, (tokens,), generator=g, device="cuda",
                                dtype=torch.int32)
    for name, e in errors(block, x, adapter_ids).items():
        print(f"{name:28s} {e:.3g}")
    y, kept = block.forward(x, adapter_ids)
    block.backward(torch.ones_like(y), kept)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(50):
        y, kept = block.forward(x, adapter_ids)
        block.backward(y, kept)
    end.record()
    torch.cuda.synchronize()
    assert q8.device_error() == 0
    took = start.elapsed_time(end) / 50 * 1e3
    print(f"forward and gradient calls of {tokens} tokens: {took:.0f} us")


if __name__ == "__main__":
    main()
