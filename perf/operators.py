"""The operators for rows of one batch that go through different weights, as
cases to measure: tokens sorted by expert and back (with gradients), the
experts' int8 products, and low-rank adapters beside a shared int8 projection.

Each case runs in two forms on the same inputs: a plain one of elementary
torch operations in 32 bits, and (``own``) this package's entry points.

kinds of case
  dispatch  slots sorted by expert and the tokens' rows gathered into that
            order; with ``grad`` also the gradient of the gather
  combine   the experts' rows weighted and added back per token; with
            ``grad`` also the gradients of the rows and of the weights
  experts   int8 rows times the int8 weight of their expert, dequantized (or
            requantized to int8)
  lora      int8 rows times one shared int8 weight, plus each row's own
            low-rank adapter
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _route(kind, name, T, k, E, H, dtype, grad=False, drop=0.0):
    return {"name": name, "kind": kind, "T": T, "k": k, "E": E, "H": H, "dtype": dtype,
            "grad": grad, "drop": drop}


def _experts(name, T, k, E, N, K, out, zp=0, bias=True, relu=False, in_order=False, drop=0.0):
    return {"name": name, "kind": "experts", "T": T, "k": k, "E": E, "N": N, "K": K, "out": out,
            "zp": zp, "bias": bias, "relu": relu, "in_order": in_order, "drop": drop}


def _lora(name, M, N, K, L, r, dtype, out, zp=0, bias=True, relu=False, runs=False, bare=0.0):
    return {"name": name, "kind": "lora", "M": M, "N": N, "K": K, "L": L, "r": r, "dtype": dtype,
            "out": out, "zp": zp, "bias": bias, "relu": relu, "runs": runs, "bare": bare}


def listed():
    return [
        # one token of a decode step, its int8 activations copied to eight experts
        _route("dispatch", "dispatch_1x8_i8", 1, 8, 64, 4096, "i8"),
        # a training batch: forward copy and the gradient that adds the copies up
        _route("dispatch", "dispatch_2048x4_bf16_grad", 2048, 4, 64, 4096, "bf16", grad=True),
        # odd sizes, padding tokens that have no expert, fp32 master activations
        _route("dispatch", "dispatch_1037x3_f32_grad", 1037, 3, 17, 1003, "f32", grad=True, drop=0.1),
        # a decode batch: eight experts' rows joined per token
        _route("combine", "combine_16x8_bf16", 16, 8, 64, 4096, "bf16"),
        # odd sizes with dropped slots, half precision, training
        _route("combine", "combine_777x5_f16_grad", 777, 5, 31, 1001, "f16", grad=True, drop=0.2),
        # a large training batch, rows far larger than the cache
        _route("combine", "combine_4096x8_bf16_grad", 4096, 8, 64, 4096, "bf16", grad=True),
        # one token of a decode step through its eight experts, int8 to int8
        _experts("experts_1x8_2048x2048_i8", 1, 8, 64, 2048, 2048, "i8", zp=-3, relu=True),
        # a decode batch: nearly every expert is read for a few rows each
        _experts("experts_16x8_2048x2048", 16, 8, 64, 2048, 2048, "bf16", zp=5),
        # a prompt: every expert multiplies hundreds of rows
        _experts("experts_2048x4_4096x4096", 2048, 4, 16, 4096, 4096, "bf16", zp=-5),
        # one request of a decode step, its own adapter
        _lora("lora_1_4096x4096_r16", 1, 4096, 4096, 8, 16, "bf16", "bf16"),
        # a decode batch of requests with many adapters, some with none
        _lora("lora_64_11008x4096_r16", 64, 11008, 4096, 32, 16, "bf16", "bf16", zp=4, bare=0.1),
        # prompts of several requests, each in one run of rows
        _lora("lora_2048_11008x4096_r64", 2048, 11008, 4096, 8, 64, "f16", "bf16", zp=-5, runs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if c["kind"] in ("experts", "lora"):
            w = work(c)
            if w["flops"] > 2.7e11 or (c["kind"] == "experts" and c["E"] * c["N"] * c["K"] > 2 ** 28):
                continue
        elif c["T"] * c["k"] * c["H"] * BYTES[c["dtype"]] > 2 ** 28:
            continue
        return c


def _draw(rng):
    kind = rng.choice(["dispatch", "combine", "experts", "lora"])
    if kind in ("dispatch", "combine"):
        E = rng.randint(4, 128)
        dtype = rng.choice(["f32", "bf16", "f16"] + (["i8"] if kind == "dispatch" else []))
        c = _route(kind, "", _log(rng, 1, 8192), rng.randint(1, min(8, E)), E,
                   _log(rng, 64, 8192) + rng.randint(0, 3), dtype,
                   grad=dtype != "i8" and rng.random() < 0.6, drop=rng.choice([0.0, 0.0, 0.15]))
    elif kind == "experts":
        E = rng.randint(4, 64)
        T, k = _log(rng, 1, 4096), rng.randint(1, min(8, E))
        c = _experts("", T, k, E, 4 * _log(rng, 64, 1024), 4 * _log(rng, 64, 1024),
                     rng.choice(["bf16", "f16", "f32", "i8"]), zp=rng.randint(-20, 20),
                     bias=rng.random() < 0.5, relu=rng.random() < 0.3,
                     in_order=rng.random() < 0.4, drop=rng.choice([0.0, 0.1]))
    else:
        c = _lora("", _log(rng, 1, 4096), 4 * _log(rng, 64, 2752), 4 * _log(rng, 64, 1024),
                  rng.randint(1, 48), rng.choice([8, 16, 16, 24, 32, 64]),
                  rng.choice(["bf16", "f16"]), rng.choice(["bf16", "f16", "f32"]),
                  zp=rng.randint(-20, 20), bias=rng.random() < 0.5, relu=rng.random() < 0.3,
                  runs=rng.random() < 0.5, bare=rng.choice([0.0, 0.2]))
    del c["name"]
    return c


def _touched(E, k, T):
    """Experts that T tokens of k distinct experts each reach, on average."""
    return E * (1.0 - (1.0 - k / E) ** T)


def work(case):
    c = case
    if c["kind"] in ("dispatch", "combine"):
        b, R = BYTES[c["dtype"]], c["T"] * c["k"]
        tokens, rows = c["T"] * c["H"] * b, R * (1.0 - c["drop"]) * c["H"] * b
        if c["kind"] == "dispatch":
            total = 12 * R + tokens + R * c["H"] * b
            if c["grad"]:
                total += rows + tokens
            return {"bytes": total, "flops": rows / b if c["grad"] else 0}
        total = 8 * R + rows + tokens
        if c["grad"]:
            total += 8 * R + rows + tokens + R * c["H"] * b  # the backward pass comes later: it reads the rows again
        return {"bytes": total, "flops": (6 if c["grad"] else 2) * rows / b}
    if c["kind"] == "experts":
        R = c["T"] * c["k"]
        kept = R * (1.0 - c["drop"])
        rows_in = R if c["in_order"] else c["T"]
        touched = _touched(c["E"], c["k"] * (1.0 - c["drop"]), c["T"])
        return {"bytes": rows_in * c["K"] + touched * c["N"] * (c["K"] + 8) + R * c["N"] * BYTES[c["out"]],
                "flops": 2.0 * kept * c["N"] * c["K"]}
    with_a = c["M"] * (1.0 - c["bare"])
    active = min(c["L"], max(1.0, _touched(c["L"], 1, with_a))) if with_a else 0
    return {"bytes": c["N"] * (c["K"] + 8) + c["M"] * c["K"] + c["M"] * c["N"] * BYTES[c["out"]]
            + active * (c["N"] + c["K"]) * c["r"] * 2,
            "flops": 2.0 * c["M"] * c["N"] * c["K"] + 2.0 * with_a * c["r"] * (c["N"] + c["K"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _routing(c, g):
    """Expert ids and weights as a router gives them: the top k of skewed scores, their softmax."""
    dev = g.device
    scores = torch.randn(c["T"], c["E"], generator=g, device=dev)
    scores += 0.7 * torch.randn(c["E"], generator=g, device=dev)
    top, ids = torch.topk(scores, c["k"], dim=1)
    ids = ids.to(torch.int32)
    if c["drop"]:
        gone = torch.rand(c["T"], c["k"], generator=g, device=dev) < c["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous(), torch.softmax(top, dim=1).contiguous()


def _sorted_slots(ids, E):
    """(order, position, offsets) of the stable sort by expert, dropped slots last and marked -1."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < E)
    key = torch.where(kept, flat, torch.full_like(flat, E))
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=flat.device))
    rows = torch.arange(flat.numel(), device=flat.device)
    position = torch.empty_like(order)
    position[order] = rows
    position = torch.where(kept, position, torch.full_like(position, -1))
    order = torch.where(rows < offsets[E], order, torch.full_like(order, -1))
    return order.int(), position.int().reshape(ids.shape), offsets.int()


def _normal(g, shape, dtype, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=g.device)).to(dtype)


def _int8(g, shape, lo, hi):
    return torch.randint(lo, hi + 1, shape, generator=g, device=g.device, dtype=torch.int8)


def _uniform(g, shape, lo, hi):
    return lo + (hi - lo) * torch.rand(shape, generator=g, device=g.device)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    if c["kind"] in ("dispatch", "combine"):
        dt = DTYPES[c["dtype"]]
        s["ids"], s["w"] = _routing(c, g)
        R = c["T"] * c["k"]
        if c["kind"] == "dispatch":
            s["x"] = _int8(g, (c["T"], c["H"]), -128, 127) if dt == torch.int8 else _normal(g, (c["T"], c["H"]), dt)
            if c["grad"]:
                s["dxs"] = _normal(g, (R, c["H"]), dt)
        else:
            s["order"], s["position"], s["offsets"] = _sorted_slots(s["ids"], c["E"])
            s["z"] = _normal(g, (R, c["H"]), dt)
            if c["grad"]:
                s["dy"] = _normal(g, (c["T"], c["H"]), dt)
        return s
    E = c["E"] if c["kind"] == "experts" else 1
    s["s_in"], s["s_out"], s["z_out"] = 0.02, 0.15, 1
    # quantized activations of a normalised layer fill the int8 range with a bell
    rows = c["T"] * (c["k"] if c["kind"] == "experts" and c["in_order"] else 1) if c["kind"] == "experts" else c["M"]
    x = torch.randn((rows, c["K"]), generator=g, device=g.device)
    s["x"] = torch.clamp(torch.round(40.0 * x) + c["zp"], -128, 127).to(torch.int8)
    s["weight"] = _int8(g, (E, c["N"], c["K"]), -127, 127)
    s["ws"] = _uniform(g, (E, c["N"]), 0.0005, 0.002) * math.sqrt(1024.0 / c["K"])
    s["b"] = 0.3 * torch.randn((E, c["N"]), generator=g, device=g.device) if c["bias"] else None
    if c["kind"] == "experts":
        s["ids"], _ = _routing(c, g)
        s["order"], s["position"], s["offsets"] = _sorted_slots(s["ids"], c["E"])
    else:
        s["ws"], s["b"] = s["ws"][0], s["b"][0] if c["bias"] else None
        dt = DTYPES[c["dtype"]]
        s["A"] = _normal(g, (c["L"], c["r"], c["K"]), dt, 1.0 / math.sqrt(c["K"]))
        s["B"] = _normal(g, (c["L"], c["N"], c["r"]), dt, 0.5 / math.sqrt(c["r"]))
        s["scaling"] = _uniform(g, (c["L"],), 0.5, 2.0)
        a = torch.randint(0, c["L"], (c["M"],), generator=g, device=g.device, dtype=torch.int32)
        if c["runs"]:
            a = torch.sort(a).values
        if c["bare"]:
            none = torch.rand(c["M"], generator=g, device=g.device) < c["bare"]
            a = torch.where(none, torch.full_like(a, -1), a)
        s["a"] = a.contiguous()
    if own:  # weights are laid out once, when a program loads them
        import int8_quantized_q8ta_gb300 as q8
        s["packed"] = q8.pack_tile_weight(s["weight"])
        if c["kind"] == "lora":
            s["adapters"] = q8.pack_lora(s["A"], s["B"], s["scaling"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_OWN if own else _PLAIN)[state["c"]["kind"]](state, state["c"])


def _own_dispatch(s, c):
    import int8_quantized_q8ta_gb300 as q8
    xs, route = q8.expert_dispatch(s["x"], s["ids"], c["E"])
    out = {"rows": xs, "order": route.order, "position": route.position, "offsets": route.offsets}
    if c["grad"]:
        out["dx"] = q8.expert_gather_backward(s["dxs"], route)
    return out


def _own_combine(s, c):
    import int8_quantized_q8ta_gb300 as q8
    route = q8.ExpertRoute(s["order"], s["position"], s["offsets"])
    out = {"y": q8.expert_combine(s["z"], s["w"], route)}
    if c["grad"]:
        out["dz"], out["dw"] = q8.expert_combine_backward(s["dy"], s["z"], s["w"], route)
    return out


def _own_experts(s, c):
    import int8_quantized_q8ta_gb300 as q8
    route = q8.ExpertRoute(s["order"], s["position"], s["offsets"])
    y = q8.linear_experts(s["x"], s["s_in"], c["zp"], s["packed"], s["ws"], s["b"], route,
                          s["s_out"], s["z_out"], activation="relu" if c["relu"] else "none",
                          x_sorted=c["in_order"], out_dtype=DTYPES[c["out"]])
    return q8.dequantize_per_tensor(y, s["s_out"], s["z_out"]) if c["out"] == "i8" else y


def _own_lora(s, c):
    import int8_quantized_q8ta_gb300 as q8
    return q8.linear_lora(s["x"], s["s_in"], c["zp"], s["packed"], s["ws"], s["b"], s["adapters"],
                          s["a"], s["s_out"], s["z_out"], activation="relu" if c["relu"] else "none",
                          out_dtype=DTYPES[c["out"]])


_OWN = {"dispatch": _own_dispatch, "combine": _own_combine, "experts": _own_experts, "lora": _own_lora}


def _plain_gather(x, order, k):
    kept = (order >= 0)[:, None]
    rows = x[(order.clamp(min=0) // k).long()]
    return torch.where(kept, rows, torch.zeros((), dtype=x.dtype, device=x.device))


def _plain_rows_of(rows, position):
    """[T, k, H] in 32 bits: each slot's sorted row, 0 where it was dropped."""
    got = rows[position.clamp(min=0).long()].float()
    return torch.where((position >= 0)[:, :, None], got, torch.zeros((), device=rows.device))


def _plain_dispatch(s, c):
    order, position, offsets = _sorted_slots(s["ids"], c["E"])
    out = {"rows": _plain_gather(s["x"], order, c["k"]), "order": order, "position": position, "offsets": offsets}
    if c["grad"]:
        out["dx"] = _plain_rows_of(s["dxs"], position).sum(1).to(s["dxs"].dtype)
    return out


def _plain_combine(s, c):
    z, w, position = s["z"], s["w"], s["position"]
    zs = _plain_rows_of(z, position)
    out = {"y": (w[:, :, None] * zs).sum(1).to(z.dtype)}
    if c["grad"]:
        dy = s["dy"].float()
        slot = s["order"].clamp(min=0).long()
        dz = w.reshape(-1)[slot][:, None] * dy[slot // c["k"]]
        out["dz"] = torch.where((s["order"] >= 0)[:, None], dz, torch.zeros((), device=z.device)).to(z.dtype)
        out["dw"] = (dy[:, None, :] * zs).sum(2)
    return out


def _finish(acc, s, c, ws, b, more=None):
    """Accumulator -> output: dequantize, bias, adapter term, activation, requantize or round."""
    v = acc * s["s_in"] * ws
    if b is not None:
        v = v + b
    if more is not None:
        v = v + more
    if c["relu"]:
        v = torch.clamp(v, min=0.0)
    if c["out"] == "i8":
        q = torch.clamp(torch.round(v * (1.0 / s["s_out"])) + s["z_out"], -128, 127)
        return (q - s["z_out"]) * s["s_out"]
    return v.to(DTYPES[c["out"]])


def _plain_experts(s, c):
    # every expert's rows in a block as high as the fullest expert's, one batched product
    order, offsets = s["order"].long(), s["offsets"].long()
    E, R = c["E"], order.numel()
    counts = offsets[1:] - offsets[:-1]
    high = max(1, int(counts.max()))
    x = (s["x"] if c["in_order"] else _plain_gather(s["x"], order, c["k"])).float() - c["zp"]
    at = offsets[:-1, None] + torch.arange(high, device=x.device)
    inside = at < offsets[1:, None]
    blocks = x[at.clamp(max=R - 1)]
    acc = torch.bmm(blocks, s["weight"].float().transpose(1, 2))
    y = _finish(acc, s, c, s["ws"][:, None, :], None if s["b"] is None else s["b"][:, None, :])
    out = torch.zeros((R, c["N"]), dtype=y.dtype, device=x.device)
    out[at[inside]] = y[inside]
    return out


def _plain_lora(s, c):
    x = s["x"].float() - c["zp"]
    L, r = c["L"], c["r"]
    acc = x @ s["weight"][0].float().t()
    mine = (s["a"][:, None] == torch.arange(L, device=x.device)) * s["scaling"]
    h = (x @ s["A"].float().reshape(L * r, -1).t()) * s["s_in"]
    h = (h.reshape(-1, L, r) * mine[:, :, None]).reshape(-1, L * r)
    more = h @ s["B"].float().transpose(1, 2).reshape(L * r, -1)
    return _finish(acc, s, c, s["ws"], s["b"], more)


_PLAIN = {"dispatch": _plain_dispatch, "combine": _plain_combine, "experts": _plain_experts, "lora": _plain_lora}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _slots64(ids, E):
    """Every kept slot's sorted row by counting: those of lower experts, and earlier ones of its own."""
    e = ids.reshape(-1).cpu().tolist()
    count = [0] * (E + 1)
    for v in e:
        if 0 <= v < E:
            count[v + 1] += 1
    for i in range(E):
        count[i + 1] += count[i]
    nxt, where = count[:], []
    for v in e:
        if 0 <= v < E:
            where.append(nxt[v])
            nxt[v] += 1
        else:
            where.append(-1)
    return torch.tensor(where, device=ids.device).reshape(ids.shape), count


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "lora":
        return _exact_lora(s, c)
    where, count = _slots64(s["ids"], c["E"])
    T, k = where.shape
    kept = where >= 0
    if c["kind"] == "experts":
        return _exact_experts(s, c, where, kept, count)
    R = T * k
    if c["kind"] == "dispatch":
        if c["dtype"] == "i8":
            return None  # whole numbers only
        rows = torch.zeros(R, c["H"], dtype=torch.float64, device=where.device)
        rows[where[kept]] = s["x"].double()[:, None, :].expand(T, k, -1)[kept]
        out = {"rows": rows, "order": None, "position": None, "offsets": None}
        if c["grad"]:
            dx = torch.zeros(T, c["H"], dtype=torch.float64, device=where.device)
            for j in range(k):
                ok = kept[:, j]
                dx[ok] += s["dxs"][where[ok, j]].double()
            out["dx"] = dx
        return out
    y = torch.zeros(T, c["H"], dtype=torch.float64, device=where.device)
    dz = torch.zeros(R, c["H"], dtype=torch.float64, device=where.device) if c["grad"] else None
    dw = torch.zeros(T, k, dtype=torch.float64, device=where.device)
    for j in range(k):
        ok = kept[:, j]
        at, w = where[ok, j], s["w"][ok, j].double()[:, None]
        z = s["z"][at].double()
        y[ok] += w * z
        if c["grad"]:
            dy = s["dy"][ok].double()
            dz[at] = w * dy
            dw[ok, j] = torch.einsum("th,th->t", dy, z)
    return {"y": y, "dz": dz, "dw": dw} if c["grad"] else {"y": y}


def _round64(v, s, c):
    if c["relu"]:
        v = v.clamp(min=0)
    if c["out"] == "i8":
        v = ((v / s["s_out"]).round() + s["z_out"]).clamp(-128, 127)
        v = (v - s["z_out"]) * s["s_out"]
    return v


def _exact_experts(s, c, where, kept, count):
    T, k = where.shape
    out = torch.zeros(T * k, c["N"], dtype=torch.float64, device=where.device)
    token = torch.empty(T * k, dtype=torch.long, device=where.device)
    token[where[kept]] = torch.arange(T, device=where.device)[:, None].expand(T, k)[kept]
    for e in range(c["E"]):
        lo, hi = count[e], count[e + 1]
        if lo == hi:
            continue
        x = s["x"][lo:hi] if c["in_order"] else s["x"][token[lo:hi]]
        v = (x.double() - c["zp"]) @ s["weight"][e].double().t() * s["s_in"] * s["ws"][e].double()
        if s["b"] is not None:
            v = v + s["b"][e].double()
        out[lo:hi] = _round64(v, s, c)
    return out


def _exact_lora(s, c):
    x = s["x"].double() - c["zp"]
    v = x @ s["weight"][0].double().t() * s["s_in"] * s["ws"].double()
    if s["b"] is not None:
        v = v + s["b"].double()
    for a in range(c["L"]):
        mine = s["a"] == a
        h = x[mine] @ s["A"][a].double().t() * s["s_in"]
        v[mine] += s["scaling"][a].double() * (h @ s["B"][a].double().t())
    return _round64(v, s, c)
