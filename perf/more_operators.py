"""Measured cases of the 8-bit operators beside the layer calls: blocks of floats quantised to e4m3
with a scale of their own, the transposed-weight product of operands held that way, and a K/V cache
that is quantised as it is written, read back, and attended by single tokens, with their gradient.

Where `own` is false every operator runs in its plain form (elementary torch operations in
32 bits); where it is true the same inputs go through this repository's library.
"""
import math

import torch

own = False

BLOCK = 128             # columns that share a scale
E4M3 = torch.float8_e4m3fn


def _tensor_type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def listed():
    """Hidden size 2560, FFN size 9728, 32 heads over 8 of 128 values, 2048 and 512 rows are the
    repository's own layer stack, 20 heads over 5 with 1024 keys its single-token layer; the others are generic."""
    return [
        # the gradient of a 2048-token sequence before a product with a frozen 8-bit weight
        {"name": "quantize_seq", "op": "quantize", "rows": 2048, "cols": 9728, "type": "f32", "block_rows": 1},
        # a frozen bf16 weight of the layer stack as a program loads it
        {"name": "quantize_weight", "op": "quantize", "rows": 2560, "cols": 9728, "type": "bf16", "block_rows": 128},
        # one token through a weight of the FFN: bound by the read of the weight
        {"name": "linear_token", "op": "linear", "rows": 1, "out": 9728, "in": 2560, "type": "f32", "add": False},
        # sizes that divide nothing, added to the other branch's gradient
        {"name": "linear_odd", "op": "linear", "rows": 333, "out": 1001, "in": 4099, "type": "f32", "add": True},
        # the 2048-token sequence through the same weight
        {"name": "linear_seq", "op": "linear", "rows": 2048, "out": 9728, "in": 2560, "type": "f32", "add": False},
        # the newest token of eight sequences into the cache: launch latency
        {"name": "write_tokens", "op": "write", "rows": 8, "slots": 16384, "kv_heads": 8, "dim": 128, "type": "bf16"},
        # keys and values of a 2048-token sequence, cached for the backward pass
        {"name": "write_seq", "op": "write", "rows": 2048, "slots": 4096, "kv_heads": 8, "dim": 128, "type": "f32"},
        # four such sequences read back for a layer call
        {"name": "read_seq", "op": "read", "rows": 8192, "slots": 16384, "kv_heads": 8, "dim": 128, "type": "f32",
         "layout": "hsd"},
        # one token over 1024 keys: the single-token layer
        {"name": "attend_token", "op": "attend", "seqs": 1, "longest": 1024, "heads": 20, "kv_heads": 5, "dim": 128,
         "page": 64, "type": "f32"},
        # a served batch, lengths between one token and 16384
        {"name": "attend_batch", "op": "attend", "seqs": 32, "longest": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "bf16"},
        # gradient of the single-token layer's attention
        {"name": "grad_token", "op": "attend_grad", "seqs": 1, "longest": 1024, "heads": 20, "kv_heads": 5, "dim": 128,
         "page": 64, "type": "f32"},
        # one long sequence: few rows, a long axis
        {"name": "grad_long", "op": "attend_grad", "seqs": 1, "longest": 131072, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "f32"},
    ]


def _log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "write", "read", "attend", "attend_grad"])
    case = {"op": op, "type": rng.choice(["f32", "bf16"])}
    if op == "quantize":
        case.update(rows=_log_between(rng, 1, 4096), cols=_log_between(rng, 16, 9728), block_rows=rng.choice([1, 128]))
    elif op == "linear":
        out, dim = _log_between(rng, 64, 9728), _log_between(rng, 64, 9728)
        if rng.random() < 0.6:                   # most weights have sizes of whole 64s
            out, dim = 64 * (out // 64), 64 * (dim // 64)
        rows = min(_log_between(rng, 1, 2048), 2048 * 9728 * 2560 // (out * dim))
        case.update(rows=rows, out=out, add=rng.random() < 0.3)
        case["in"] = dim
    else:
        kv_heads, dim = rng.choice([1, 2, 5, 8]), rng.choice([64, 96, 128, 256])
        if op in ("write", "read"):
            rows = _log_between(rng, 1, 4096)
            case.update(rows=rows, slots=rows + _log_between(rng, 1, 4096), kv_heads=kv_heads, dim=dim)
            if op == "read":
                case["layout"] = rng.choice(["shd", "hsd"])
        else:
            seqs = _log_between(rng, 1, 64)
            # no more keys in all than the batch (attend) or the long sequence (attend_grad) that are listed
            most = (32 * 16384 if op == "attend" else 131072) * 8 * 128 // (seqs * kv_heads * dim)
            case.update(seqs=seqs, longest=_log_between(rng, 1, min(most, 65536)), kv_heads=kv_heads, dim=dim,
                        heads=kv_heads * rng.choice([1, 3, 4, 8]), page=rng.choice([1, 16, 64, 100]))
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _scales(x, block_rows):
    """The smallest power of two by which each block fits e4m3's 448: [blocks of rows, blocks of columns]."""
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK, 0, -rows % block_rows))
    top = pad.reshape(-(-rows // block_rows), block_rows, -(-cols // BLOCK), BLOCK).abs().amax((1, 3))
    bits = top.view(torch.int32)
    power = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=1)    # 448 = 1.75 x 2^8
    return torch.where(top.isfinite(), (power << 23).view(torch.float32), torch.full_like(top, math.nan))


def _spread(scales, block_rows, rows, cols):
    """The scale of every element of a [rows, cols] matrix."""
    return scales.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def _quantized(x, block_rows):
    scales = _scales(x, block_rows)
    return (x.float() / _spread(scales, block_rows, *x.shape)).to(E4M3), scales


def _gradient_rows(gen, rows, cols):
    """Rows of gradients: their sizes differ from token to token and they have a few large columns."""
    size = torch.exp(torch.randn(rows, 1, generator=gen, device="cuda") * 2.0 - 6.0)
    columns = 1.0 + 9.0 * (torch.rand(1, cols, generator=gen, device="cuda") < 0.01)
    return torch.randn(rows, cols, generator=gen, device="cuda") * size * columns


def _quantize_inputs(case, seed):
    gen = _generator(seed)
    if case["block_rows"] == 1:
        x = _gradient_rows(gen, case["rows"], case["cols"])
    else:
        x = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda") * 0.02
    return x.to(_tensor_type(case["type"]))


def _linear_inputs(case, seed):
    """An 8-bit weight [in, out] whose scales are any floats (as where amax / 448 was taken), rows of
    quantised gradients, and what the product is added to."""
    gen = _generator(seed)
    weight, w_scales = _quantized(torch.randn(case["in"], case["out"], generator=gen, device="cuda") * 0.02, BLOCK)
    w_scales = w_scales * (0.6 + 0.4 * torch.rand(w_scales.shape, generator=gen, device="cuda"))
    grad, g_scales = _quantized(_gradient_rows(gen, case["rows"], case["out"]), 1)
    base = torch.randn(case["rows"], case["in"], generator=gen, device="cuda").to(_tensor_type(case["type"]))
    return weight, w_scales, grad, g_scales, base


def _cache_inputs(gen, slots, kv_heads, dim):
    """A filled cache: e4m3 rows [slots, kv_heads, dim] of keys (their heads of different size) and values, and
    their scales [kv_heads, slots]."""
    size = torch.exp(torch.randn(1, kv_heads, 1, generator=gen, device="cuda") * 0.3)
    k = torch.randn(slots, kv_heads, dim, generator=gen, device="cuda") * size
    v = torch.randn(slots, kv_heads, dim, generator=gen, device="cuda")
    return _cached(k) + _cached(v)


def _cached(rows):
    """Rows [n, kv_heads, dim] as the cache holds them: one scale a row and head."""
    top = rows.float().abs().amax(2)
    bits = top.view(torch.int32)
    power = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000)).clamp(min=1)
    scale = torch.where(top.isfinite(), (power << 23).view(torch.float32), torch.full_like(top, math.nan))
    return (rows.float() / scale[:, :, None]).to(E4M3), scale.T.contiguous()


def _rows_inputs(case, seed):
    """A cache, the slots of some rows in no order (where they are read, one in fifty left out, as padding is), and new rows."""
    gen = _generator(seed)
    cache = _cache_inputs(gen, case["slots"], case["kv_heads"], case["dim"])
    slots = torch.randperm(case["slots"], generator=gen, device="cuda")[:case["rows"]]
    if case["op"] == "read":
        padding = torch.rand(case["rows"], generator=gen, device="cuda") < 0.02
        slots = torch.where(padding, torch.full_like(slots, -1), slots)
    new = [torch.randn(case["rows"], case["kv_heads"], case["dim"], generator=gen, device="cuda")
           .to(_tensor_type(case["type"])) for _ in range(2)]
    return cache, slots, new


def _attend_inputs(case, seed):
    """A cache whose pages lie in no order, sequences of different lengths (the longest among them), a query
    for each sequence's newest token and the gradient of what it attends to."""
    gen = _generator(seed)
    seqs, page = case["seqs"], case["page"]
    spread = torch.rand(seqs, generator=gen, device="cuda")
    lengths = torch.exp(spread * math.log(case["longest"])).round().to(torch.int32)
    lengths[0] = case["longest"]
    most = -(-case["longest"] // page)
    pages = torch.randperm(seqs * most, generator=gen, device="cuda").to(torch.int32).reshape(seqs, most)
    cache = _cache_inputs(gen, seqs * most * page, case["kv_heads"], case["dim"])
    kind = _tensor_type(case["type"])
    q = torch.randn(seqs, case["heads"], case["dim"], generator=gen, device="cuda").to(kind)
    d_ctx = (torch.randn(seqs, case["heads"], case["dim"], generator=gen, device="cuda") * 0.1).to(kind)
    return cache, pages, lengths, q, d_ctx


def prepare(case, seed):
    state = {"case": case}
    if case["op"] == "quantize":
        state["x"] = _quantize_inputs(case, seed)
        return state
    if case["op"] == "linear":
        state["weight"], state["w_scales"], state["grad"], state["g_scales"], state["out"] = _linear_inputs(case, seed)
        if own:
            import transformer_layer_backward_gb300 as tlb
            state["ws"] = tlb.linear_fp8_workspace(case["rows"], case["out"], case["in"])
        return state
    if case["op"] in ("write", "read"):
        state["cache"], state["slots"], state["new"] = _rows_inputs(case, seed)
    else:
        state["cache"], state["pages"], state["lengths"], state["q"], state["d_ctx"] = _attend_inputs(case, seed)
        if case["op"] == "attend_grad":
            state["lse"] = _plain_attend(case, state)[1]["lse"]
    if own:
        import transformer_layer_backward_gb300 as tlb
        state["handle"] = tlb.kv8_cache_of(*state["cache"])
        if case["op"] in ("attend", "attend_grad"):
            state["ws"] = tlb.kv8_attn_workspace(state["handle"], case["seqs"], case["heads"], case["longest"],
                                                 grad=case["op"] == "attend_grad")
    return state


# ---------------------------------------------------------------- one pass

def _plain_linear(case, state):
    weight = state["weight"].float() * _spread(state["w_scales"], BLOCK, case["in"], case["out"])
    grad = state["grad"].float() * _spread(state["g_scales"], 1, case["rows"], case["out"])
    product = grad @ weight.T
    if case["add"]:
        product = product + state["out"].float()
    return product.to(_tensor_type(case["type"]))


def _plain_write(state):
    (k, k_scale, v, v_scale), slots, new = state["cache"], state["slots"], state["new"]
    for rows, values, scales in ((new[0], k, k_scale), (new[1], v, v_scale)):
        codes, scale = _cached(rows)
        values.view(torch.uint8)[slots] = codes.view(torch.uint8)
        scales[:, slots] = scale
    return {"k": k, "k_scale": k_scale, "v": v, "v_scale": v_scale}


def _plain_read(case, state):
    k, k_scale, v, v_scale = state["cache"]
    slots = state["slots"]
    at, there = slots.clamp(min=0), (slots >= 0)[:, None, None]
    out = {}
    for name, values, scales in (("k", k, k_scale), ("v", v, v_scale)):
        rows = values.view(torch.uint8)[at].view(E4M3).float() * scales[:, at].T[:, :, None]
        rows = torch.where(there, rows, torch.zeros_like(rows)).to(_tensor_type(case["type"]))
        out[name] = rows.transpose(0, 1).contiguous() if case["layout"] == "hsd" else rows
    return out


def _gathered(case, state):
    """Every sequence's keys and values [seqs, kv_heads, longest, dim] in 32 bits, and which of them are there."""
    k, k_scale, v, v_scale = state["cache"]
    j = torch.arange(case["longest"], device="cuda")
    at = state["pages"].long()[:, j // case["page"]] * case["page"] + j % case["page"]
    there = j[None, :] < state["lengths"][:, None]
    rows = [(values.view(torch.uint8)[at].view(E4M3).float() * scales.T[at][..., None]).transpose(1, 2)
            for values, scales in ((k, k_scale), (v, v_scale))]
    return rows[0], rows[1], there[:, None, None, :]


def _grouped(case, x):
    return x.float().reshape(case["seqs"], case["kv_heads"], -1, case["dim"])


def _plain_attend(case, state):
    k, v, there = _gathered(case, state)
    logits = _grouped(case, state["q"]) @ k.mT / math.sqrt(case["dim"])
    logits = logits.masked_fill(~there, -math.inf)
    top = logits.amax(3, keepdim=True)
    weights = (logits - top).exp()
    total = weights.sum(3, keepdim=True)
    ctx = (weights / total) @ v
    lse = (top + total.log())[..., 0].reshape(case["seqs"], case["heads"])
    return (k, v, there), {"ctx": ctx.reshape(state["q"].shape).to(state["q"].dtype), "lse": lse}


def _plain_attend_grad(case, state):
    k, v, there = _gathered(case, state)
    q, d_ctx = _grouped(case, state["q"]), _grouped(case, state["d_ctx"])
    scale = 1.0 / math.sqrt(case["dim"])
    logits = (q @ k.mT * scale).masked_fill(~there, -math.inf)
    p = (logits - state["lse"].reshape(*q.shape[:3], 1)).exp()
    d_p = d_ctx @ v.mT
    d_s = p * (d_p - (p * d_p).sum(3, keepdim=True))
    d_q = d_s @ k * scale
    newest = (state["lengths"].long() - 1)[:, None, None, None].expand(*q.shape[:3], 1)
    d_k = (d_s.gather(3, newest) * q).sum(2) * scale
    d_v = (p.gather(3, newest) * d_ctx).sum(2)
    kind = state["q"].dtype
    return {"d_q": d_q.reshape(state["q"].shape).to(kind), "d_k": d_k.to(kind), "d_v": d_v.to(kind)}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import transformer_layer_backward_gb300 as tlb
        if op == "quantize":
            values, scales = tlb.fp8_quantize(state["x"], block_rows=case["block_rows"])
            return {"values": values, "scales": scales}
        if op == "linear":
            out = state["out"].clone() if case["add"] else None
            return {"d_x": tlb.linear_fp8_backward(state["weight"], state["w_scales"], state["grad"], state["g_scales"],
                                                   out=out, accumulate=case["add"], dtype=_tensor_type(case["type"]),
                                                   ws=state["ws"])}
        if op == "write":
            tlb.kv8_write(state["handle"], *state["new"], state["slots"])
            k, k_scale, v, v_scale = state["cache"]
            return {"k": k, "k_scale": k_scale, "v": v, "v_scale": v_scale}
        if op == "read":
            k, v = tlb.kv8_read(state["handle"], state["slots"], dtype=_tensor_type(case["type"]), kv_layout=case["layout"])
            return {"k": k, "v": v}
        over = (state["handle"], state["q"], state["pages"], case["page"], state["lengths"], case["longest"])
        if op == "attend":
            ctx, lse = tlb.kv8_attn_forward(*over, ws=state["ws"])
            return {"ctx": ctx, "lse": lse}
        d_q, d_k, d_v = tlb.kv8_attn_backward(*over, state["lse"], state["d_ctx"], ws=state["ws"])
        return {"d_q": d_q, "d_k": d_k, "d_v": d_v}
    if op == "quantize":
        values, scales = _quantized(state["x"], case["block_rows"])
        return {"values": values, "scales": scales}
    if op == "linear":
        return {"d_x": _plain_linear(case, state)}
    if op == "write":
        return _plain_write(state)
    if op == "read":
        return _plain_read(case, state)
    return _plain_attend(case, state)[1] if op == "attend" else _plain_attend_grad(case, state)


def work(case):
    wide = {"bf16": 2, "f32": 4}[case["type"]]
    if case["op"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        blocks = -(-rows // case["block_rows"]) * -(-cols // BLOCK)
        return {"bytes": rows * cols * (wide + 1) + blocks * 4, "flops": 2 * rows * cols}
    if case["op"] == "linear":
        rows, out, dim = case["rows"], case["out"], case["in"]
        columns = -(-out // BLOCK)
        size = rows * out + dim * out + (rows + -(-dim // BLOCK)) * columns * 4
        return {"bytes": size + rows * dim * wide * (3 if case["add"] else 1), "flops": 2 * rows * out * dim}
    per_row = case["kv_heads"] * (case["dim"] + 4)               # one key or value row of the cache
    if case["op"] in ("write", "read"):
        return {"bytes": case["rows"] * (8 + 2 * (per_row + case["kv_heads"] * case["dim"] * wide)),
                "flops": 2 * case["rows"] * case["kv_heads"] * case["dim"]}
    # lengths are spread evenly over their logarithm: this is their mean, the longest counted for itself
    seqs, longest = case["seqs"], case["longest"]
    keys = longest + (seqs - 1) * ((longest - 1) / math.log(longest) if longest > 1 else 1)
    tokens = seqs * case["heads"] * case["dim"] * wide
    products = 2 if case["op"] == "attend" else 3
    return {"bytes": 2 * keys * per_row + 2 * tokens + (0 if products == 2 else tokens + 2 * tokens // case["heads"] * case["kv_heads"])
            + seqs * case["heads"] * 4, "flops": 2 * products * keys * case["heads"] * case["dim"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_blocks(x, block_rows, block):
    """Each value over the smallest power of two that brings its block within 448, rounded to 3 bits after the
    leading one (ties to even), in steps of 2^-9 at least; and those powers."""
    rows, cols = x.shape
    padded = torch.zeros(-(-rows // block_rows) * block_rows, -(-cols // block) * block, dtype=torch.float64, device="cuda")
    padded[:rows, :cols] = x.abs()
    top = padded.unfold(0, block_rows, block_rows).unfold(1, block, block).amax((2, 3))
    power = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0)
    r, c = torch.arange(rows, device="cuda") // block_rows, torch.arange(cols, device="cuda") // block
    value = x.double() / torch.exp2(power)[r][:, c]
    step = torch.exp2(torch.floor(torch.log2(value.abs())).clamp(min=-6.0) - 3.0)
    return torch.round(value / step) * step, torch.exp2(power)


def _exact_rows(rows):
    values, scales = _exact_blocks(rows.reshape(-1, rows.shape[-1]), 1, rows.shape[-1])
    return values.reshape(rows.shape), scales.reshape(rows.shape[:2]).T


def _exact_linear(case, seed):
    weight, w_scales, grad, g_scales, base = _linear_inputs(case, seed)
    out = base.double() if case["add"] else torch.zeros(base.shape, dtype=torch.float64, device="cuda")
    for start in range(0, case["out"], BLOCK):
        g = grad[:, start:start + BLOCK].double() * g_scales[:, start // BLOCK, None].double()
        w = weight[:, start:start + BLOCK].double()
        w = w * w_scales[torch.arange(case["in"], device="cuda") // BLOCK, start // BLOCK, None].double()
        out = out + g @ w.T
    return {"d_x": out}


def _exact_attention(case, seed, grad):
    (k, k_scale, v, v_scale), pages, lengths, q, d_ctx = _attend_inputs(case, seed)
    group, scale = case["heads"] // case["kv_heads"], case["dim"] ** -0.5
    found = []
    for b in range(case["seqs"]):
        n = int(lengths[b])
        j = torch.arange(n, device="cuda")
        at = pages[b].long()[torch.div(j, case["page"], rounding_mode="floor")] * case["page"] + torch.remainder(j, case["page"])
        keys = k.view(torch.uint8)[at].view(E4M3).double() * k_scale[:, at].T.double()[..., None]
        values = v.view(torch.uint8)[at].view(E4M3).double() * v_scale[:, at].T.double()[..., None]
        heads = q[b].double().unflatten(0, (case["kv_heads"], group))
        logits = torch.einsum("kgd,nkd->kgn", heads, keys) * scale
        lse = torch.logsumexp(logits, 2)
        p = torch.exp(logits - lse[..., None])
        if not grad:
            found.append((torch.einsum("kgn,nkd->kgd", p, values).flatten(0, 1), lse.flatten()))
            continue
        d = d_ctx[b].double().unflatten(0, (case["kv_heads"], group))
        d_p = torch.einsum("kgd,nkd->kgn", d, values)
        d_s = p * (d_p - (p * d_p).sum(2, keepdim=True)) * scale
        found.append((torch.einsum("kgn,nkd->kgd", d_s, keys).flatten(0, 1),
                      torch.einsum("kg,kgd->kd", d_s[..., -1], heads), torch.einsum("kg,kgd->kd", p[..., -1], d)))
    return dict(zip(("d_q", "d_k", "d_v") if grad else ("ctx", "lse"), (torch.stack(x) for x in zip(*found))))


def exact(case, seed):
    op = case["op"]
    if op == "quantize":
        values, scales = _exact_blocks(_quantize_inputs(case, seed), case["block_rows"], BLOCK)
        return {"values": values, "scales": scales}
    if op == "linear":
        return _exact_linear(case, seed)
    if op in ("attend", "attend_grad"):
        return _exact_attention(case, seed, op == "attend_grad")
    (k, k_scale, v, v_scale), slots, new = _rows_inputs(case, seed)
    if op == "write":
        out = {"k": k.double(), "k_scale": k_scale.double(), "v": v.double(), "v_scale": v_scale.double()}
        for name, rows in zip("kv", new):
            values, scales = _exact_rows(rows)
            out[name][slots], out[name + "_scale"][:, slots] = values, scales
        return out
    out = {}
    for name, values, scales in (("k", k, k_scale), ("v", v, v_scale)):
        rows = torch.zeros(case["rows"], case["kv_heads"], case["dim"], dtype=torch.float64, device="cuda")
        there = slots >= 0
        rows[there] = values.double()[slots[there]] * scales.double().T[slots[there]][..., None]
        out[name] = rows.permute(1, 0, 2).contiguous() if case["layout"] == "hsd" else rows
    return out
