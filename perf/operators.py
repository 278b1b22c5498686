"""Measured cases of the operators around the layer stack: the loss of a linear head over a
vocabulary, its gradient, and the Muon step of LoRA adapters.

Where `own` is false every operator runs in its plain form (elementary torch operations in
32 bits); where it is true the same inputs go through this repository's library.
"""
import functools
import math

import torch

own = False

#: share of the token rows that carry no target (prompt tokens and padding)
NO_TARGET = 0.1


def _tensor_type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def listed():
    """Hidden size 2560, 2048 rows, ranks 16 and 36 layers are the repository's own layer
    stack; vocabulary sizes are generic (powers of two and one prime)."""
    head = {"op": "xent_forward"}
    grad = {"op": "xent_backward", "grad_w": False}
    return [
        # loss of one token: scoring while decoding, bound by the read of the head
        {"name": "fwd_token", **head, "rows": 1, "dim": 2560, "vocab": 32768, "hidden": "bf16", "weight": "bf16"},
        # a float32 model with sizes that divide nothing, as a small or pruned head has
        {"name": "fwd_odd_f32", **head, "rows": 333, "dim": 1001, "vocab": 50021, "hidden": "f32", "weight": "f32"},
        # evaluation of one 2048-token sequence over a large vocabulary
        {"name": "fwd_seq", **head, "rows": 2048, "dim": 2560, "vocab": 131072, "hidden": "bf16", "weight": "bf16"},
        # gradient of one token: the single-token layer backward's dOut
        {"name": "bwd_token", **grad, "rows": 1, "dim": 2560, "vocab": 32768, "hidden": "bf16", "weight": "bf16"},
        # float32 activations on a bf16 head, as the layer stack keeps them: dOut of a 512-token sequence
        {"name": "bwd_seq512_f32", **grad, "rows": 512, "dim": 2560, "vocab": 32768, "hidden": "f32", "weight": "bf16"},
        # a trained head with ragged sizes: the gradient of the head too
        {"name": "bwd_odd_head", **grad, "grad_w": True, "rows": 777, "dim": 1000, "vocab": 50021, "hidden": "bf16",
         "weight": "bf16"},
        # the frozen head above the 2048-token layer stack
        {"name": "bwd_seq", **grad, "rows": 2048, "dim": 2560, "vocab": 131072, "hidden": "bf16", "weight": "bf16"},
        # the largest: two 2048-token sequences and a head that is trained too
        {"name": "bwd_large_head", **grad, "grad_w": True, "rows": 4096, "dim": 2560, "vocab": 65536, "hidden": "bf16",
         "weight": "bf16"},
        # one adapter matrix by itself: launch latency
        {"name": "muon_one", "op": "muon", "groups": "1x16x2560", "nesterov": True, "steps": 5},
        # every adapter of a 36-layer stack in one call (A of Q and V, B of Q, B of V)
        {"name": "muon_stack", "op": "muon", "groups": "72x16x2560 36x4096x16 36x1024x16", "nesterov": True, "steps": 5},
        # small odd adapters, wide and tall
        {"name": "muon_odd", "op": "muon", "groups": "7x5x1001 3x999x33", "nesterov": False, "steps": 5},
        # the same stack at the largest rank
        {"name": "muon_rank64", "op": "muon", "groups": "72x64x2560 36x4096x64 36x1024x64",
         "nesterov": True, "steps": 5},
    ]


def _log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["xent_forward", "xent_backward", "muon"])
    if op == "muon":
        groups = []
        for _ in range(rng.randint(1, 3)):
            rank, length = _log_between(rng, 1, 64), _log_between(rng, 64, 9728)
            groups.append("%dx%dx%d" % ((_log_between(rng, 1, 36),) + ((rank, length) if rng.random() < 0.5 else (length, rank))))
        return {"op": op, "groups": " ".join(groups), "nesterov": rng.random() < 0.5, "steps": rng.randint(3, 6)}
    dim, vocab = _log_between(rng, 64, 4096), _log_between(rng, 1000, 131072)
    if rng.random() < 0.5:                       # half of the heads have sizes of whole 64s
        dim, vocab = 64 * max(1, dim // 64), 64 * (vocab // 64)
    most = 2048 * 2560 * 131072
    case = {"op": op, "rows": min(_log_between(rng, 1, 4096), most // (dim * vocab)), "dim": dim, "vocab": vocab,
            "hidden": rng.choice(["bf16", "bf16", "f32"]), "weight": "bf16"}
    if case["hidden"] == "f32" and rng.random() < 0.5:
        case["weight"] = "f32"
    if op == "xent_backward":
        case["grad_w"] = rng.random() < 0.4
    return case


# ---------------------------------------------------------------- inputs

def _groups(case):
    """"36x4096x16 ..." as (count, rows, cols) of each group of adapter matrices."""
    return [tuple(int(n) for n in group.split("x")) for group in case["groups"].split()]


def _head_inputs(case, seed):
    """Hidden rows after a final norm (unit variance, plus a pull towards the target's row of
    the head of a strength between none and certain), a head of std 0.02, targets with some
    rows left out, and per-token weights of the loss."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, dim, vocab = case["rows"], case["dim"], case["vocab"]
    weight = (torch.randn(vocab, dim, generator=gen, device="cuda") * 0.02).to(_tensor_type(case["weight"]))
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    pull = torch.rand(rows, 1, generator=gen, device="cuda") * 12.0
    towards = weight[targets].float()
    towards = towards / (towards.square().sum(1, keepdim=True) + 1e-12)
    hidden = (torch.randn(rows, dim, generator=gen, device="cuda") + pull * towards).to(_tensor_type(case["hidden"]))
    left_out = torch.rand(rows, generator=gen, device="cuda") < NO_TARGET
    left_out[0] = False
    targets = torch.where(left_out, torch.full_like(targets, -1), targets)
    d_loss = (torch.rand(rows, generator=gen, device="cuda") + 0.5) / rows
    return hidden, weight, targets, d_loss


def _lse(hidden, weight):
    """The row statistics that a loss call leaves for the gradient."""
    return torch.logsumexp(hidden.float() @ weight.float().T, 1)


def _muon_inputs(case, seed):
    """Parameters of std 0.02, gradients and momenta whose singular values fall by a factor of
    100 over the rank (adapter gradients are far from orthogonal), per group [count, rows, cols]."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def falling(count, rows, cols):
        side = min(rows, cols)
        fall = torch.logspace(0.0, -2.0, side, device="cuda")
        left = torch.randn(count, rows, side, generator=gen, device="cuda")
        right = torch.randn(count, side, cols, generator=gen, device="cuda")
        return (left * fall) @ right / math.sqrt(side)

    return [(torch.randn(*g, generator=gen, device="cuda") * 0.02, falling(*g), falling(*g)) for g in _groups(case)]


MUON = {"lr": 0.02, "momentum": 0.95, "weight_decay": 0.01, "eps": 1e-7, "coefficients": (3.4445, -4.7750, 2.0315)}


def prepare(case, seed):
    if case["op"] == "muon":
        state = {"case": case, "groups": _muon_inputs(case, seed)}
        if own:
            import transformer_layer_backward_gb300 as tlb
            state["mats"] = tlb.muon_mats(*([m for group in state["groups"] for m in group[i].unbind(0)]
                                            for i in range(3)))
            state["cfg"] = tlb.muon_cfg(MUON["lr"], MUON["momentum"], MUON["weight_decay"], MUON["eps"],
                                        MUON["coefficients"], case["steps"], case["nesterov"])
            state["ws"] = tlb.muon_workspace(state["mats"])
        return state
    hidden, weight, targets, d_loss = _head_inputs(case, seed)
    state = {"case": case, "hidden": hidden, "weight": weight, "targets": targets, "d_loss": d_loss}
    if case["op"] == "xent_backward":
        state["lse"] = _lse(hidden, weight)
    if own:
        import transformer_layer_backward_gb300 as tlb
        state["ws"] = tlb.xent_workspace(hidden.dtype, weight.dtype, case["rows"], case["vocab"], case["dim"],
                                         grad_w=case.get("grad_w", False))
    return state


# ---------------------------------------------------------------- one pass

def _plain_forward(hidden, weight, targets):
    logits = hidden.float() @ weight.float().T
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    at = logits.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(targets >= 0, lse - at, torch.zeros_like(lse)), "lse": lse}


def _plain_backward(hidden, weight, targets, lse, d_loss, grad_w):
    wide_h, wide_w = hidden.float(), weight.float()
    d_logits = (wide_h @ wide_w.T - lse[:, None]).exp()
    d_logits[torch.arange(len(targets), device=targets.device), targets.clamp(min=0)] -= 1.0
    d_logits = d_logits * torch.where(targets >= 0, d_loss, torch.zeros_like(d_loss))[:, None]
    out = {"d_hidden": (d_logits @ wide_w).to(hidden.dtype)}
    if grad_w:
        out["d_weight"] = (d_logits.T @ wide_h).to(hidden.dtype)
    return out


def _scale(rows, cols):
    return math.sqrt(max(1.0, rows / cols))


def _newton_schulz(x, coefficients):
    a, b, c = coefficients
    gram = x @ x.mT
    return a * x + (b * gram + c * (gram @ gram)) @ x


def _plain_muon(param, grad, momentum, steps, nesterov):
    """One Muon step in place on a [count, rows, cols] group."""
    momentum.mul_(MUON["momentum"]).add_(grad)
    update = grad + MUON["momentum"] * momentum if nesterov else momentum
    rows, cols = update.shape[1:]
    x = update.mT if rows > cols else update
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + MUON["eps"])
    x = functools.reduce(_newton_schulz, [MUON["coefficients"]] * steps, x)
    x = x.mT if rows > cols else x
    param.sub_(MUON["lr"] * (MUON["weight_decay"] * param + _scale(rows, cols) * x))
    return param, momentum


def run(state):
    case = state["case"]
    if own:
        import transformer_layer_backward_gb300 as tlb
        if case["op"] == "muon":
            tlb.muon(state["mats"], state["cfg"], state["ws"])
            return [(param, momentum) for param, _, momentum in state["groups"]]
        hidden, weight, targets, ws = state["hidden"], state["weight"], state["targets"], state["ws"]
        if case["op"] == "xent_forward":
            loss, lse = tlb.xent_forward(hidden, weight, targets, ws=ws)
            return {"loss": loss, "lse": lse}
        d_hidden, d_weight = tlb.xent_backward(hidden, weight, targets, state["lse"], state["d_loss"],
                                               grad_w=case["grad_w"], ws=ws)
        return {"d_hidden": d_hidden, "d_weight": d_weight} if case["grad_w"] else {"d_hidden": d_hidden}
    if case["op"] == "muon":
        return [_plain_muon(*group, case["steps"], case["nesterov"]) for group in state["groups"]]
    if case["op"] == "xent_forward":
        return _plain_forward(state["hidden"], state["weight"], state["targets"])
    return _plain_backward(state["hidden"], state["weight"], state["targets"], state["lse"], state["d_loss"],
                           case["grad_w"])


def work(case):
    if case["op"] == "muon":
        size = flops = 0
        for count, rows, cols in _groups(case):
            side, length = min(rows, cols), max(rows, cols)
            size += count * rows * cols * 4 * 5                     # p, g, m read; p, m written
            # the Gram matrix (symmetric), the iteration on it, and its product with the update
            flops += count * (side * (side + 1) * length + case["steps"] * 4 * side ** 3 + 2 * side * side * length)
        return {"bytes": size, "flops": flops}
    rows, dim, vocab = case["rows"], case["dim"], case["vocab"]
    wide = {"bf16": 2, "f32": 4}
    size = rows * dim * wide[case["hidden"]] + vocab * dim * wide[case["weight"]] + rows * 16     # targets, two floats
    products = 1
    if case["op"] == "xent_backward":
        size += rows * dim * wide[case["hidden"]]
        products = 2
        if case["grad_w"]:
            size += vocab * dim * wide[case["hidden"]]
            products = 3
    return {"bytes": size, "flops": 2 * products * rows * dim * vocab}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_muon(case, seed):
    a, b, c = MUON["coefficients"]
    out = []
    for param, grad, momentum in _muon_inputs(case, seed):
        param, grad, momentum = param.double(), grad.double(), momentum.double()
        momentum = grad + momentum * MUON["momentum"]
        x = grad + momentum * MUON["momentum"] if case["nesterov"] else momentum
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + MUON["eps"])
        for _ in range(case["steps"]):
            # with x = U S V^T each step maps a singular value s to a s + b s^3 + c s^5
            cube = torch.bmm(torch.bmm(x, x.transpose(1, 2)), x) if x.shape[1] <= x.shape[2] else \
                torch.bmm(x, torch.bmm(x.transpose(1, 2), x))
            fifth = torch.bmm(torch.bmm(cube, x.transpose(1, 2)), x) if x.shape[1] <= x.shape[2] else \
                torch.bmm(cube, torch.bmm(x.transpose(1, 2), x))
            x = a * x + b * cube + c * fifth
        step = MUON["lr"] * _scale(x.shape[1], x.shape[2])
        out.append((param * (1.0 - MUON["lr"] * MUON["weight_decay"]) - step * x, momentum))
    return out


def exact(case, seed):
    if case["op"] == "muon":
        return _exact_muon(case, seed)
    hidden, weight, targets, d_loss = _head_inputs(case, seed)
    wide = hidden.double()
    has = targets >= 0
    piece = 8192
    if case["op"] == "xent_forward":
        parts, at = [], torch.zeros(len(targets), dtype=torch.float64, device="cuda")
        for start in range(0, case["vocab"], piece):
            logits = wide @ weight[start:start + piece].double().T
            parts.append(torch.logsumexp(logits, 1))
            here = (targets >= start) & (targets < start + piece)
            at[here] = logits[here, targets[here] - start]
        lse = torch.logsumexp(torch.stack(parts, 1), 1)
        return {"loss": (lse - at) * has, "lse": lse}
    lse = _lse(hidden, weight).double()
    d_hidden, d_weight = torch.zeros_like(wide), []
    for start in range(0, case["vocab"], piece):
        w = weight[start:start + piece].double()
        grad = torch.exp(wide @ w.T - lse[:, None])
        here = (targets >= start) & (targets < start + piece)
        grad[here, targets[here] - start] -= 1.0
        grad = grad * (d_loss.double() * has)[:, None]
        d_hidden += grad @ w
        if case["grad_w"]:
            d_weight.append(grad.T @ wide)
    return {"d_hidden": d_hidden, "d_weight": torch.cat(d_weight)} if case["grad_w"] else {"d_hidden": d_hidden}
