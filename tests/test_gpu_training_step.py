"""A whole fine-tuning step as it is used: the loss of the head on the final-norm output, its
gradient, back through the final RMSNorm, the layer stack (its AdamW off: lr 0), and the Muon
step of every adapter; eager and as one captured graph, against the float64 oracle.

Tolerances: the stated bars of the layer paths (float32 1e-5, tensor-core bf16 5e-3) on the
gradients.  The Muon update is compared through the step's own gradients (a weak direction of
a gradient that is itself 5e-3 off may point anywhere), to 2.5e-5 as in its own tests.
"""
import numpy as np
import pytest

from oracle import layer as OL
from oracle import ops
from synth import SEQ512, TINY, layer_inputs, rng
from tests.helpers import BF16_REL_L2, adam_to_abi, cfg_to_abi, check, host
from tests.test_gpu_muon import COEF, UPDATE_REL
from tests.test_gpu_stack import device_stack

pytestmark = pytest.mark.gpu


def normal(name, shape, std=1.0):
    n = int(np.prod(shape))
    return rng.normal(rng.stream_key(0, "step", name, *shape), n, 0.0, std).reshape(shape).astype(np.float32)


def config(kind):
    if kind == "tiny":
        return TINY.with_(name="tiny_step", n_layers=2, lr=0.0)
    return SEQ512.with_(name="seq_step", dim=512, ffn_dim=1024, n_heads=8, n_kv_heads=2, head_dim=64, rank=16,
                        lora_alpha=32.0, seq_len=200, cache_len=200, n_layers=2, lr=0.0)


@pytest.mark.parametrize("kind", ["tiny", "bf16"])
def test_training_step(lib, kind):
    import torch
    cfg, vocab, eps = config(kind), 1003, 1e-6
    S, L, n = cfg.seq_len, cfg.cache_len, cfg.n_layers
    layers = [layer_inputs(cfg, layer=l, seed=8, with_dout=False) for l in range(n)]
    x, gamma = normal("x", (S, cfg.dim)), rng.uniform(rng.stream_key(0, "step", "gamma"), cfg.dim, 0.5, 1.5).astype(np.float32)
    hidden = (x / np.sqrt(np.mean(x.astype(np.float64) ** 2, 1, keepdims=True) + eps) * gamma).astype(np.float32)
    head = normal("head", (vocab, cfg.dim), 0.1)
    targets = np.random.default_rng(0).integers(0, vocab, S)
    targets[: S // 4] = -1                                     # the prompt
    d_loss = np.full(S, 1.0 / np.sum(targets >= 0), np.float32)

    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    th, tx, tg, tt, td = dev(hidden), dev(x), dev(gamma), dev(targets), dev(d_loss)
    tw = dev(head) if kind == "tiny" else dev(head).bfloat16()
    c, adam = cfg_to_abi(lib, cfg), adam_to_abi(lib, cfg)
    devs = device_stack(lib, cfg, layers, with_grads=True)
    names = ("a_q", "b_q", "a_v", "b_v")
    params = [d["L"][k] for d in devs for k in names]
    grads = [d["g"]["d" + k[0].upper() + k[1:]] for d in devs for k in names]
    momenta = [torch.zeros_like(p) for p in params]
    before = [p.clone() for p in params]
    mats = lib.muon_mats(params, grads, momenta)
    mcfg = lib.muon_cfg(0.02, weight_decay=0.01)
    ws_x = lib.xent_workspace(th.dtype, tw.dtype, S, vocab, cfg.dim)
    ws_s, ws_m = lib.stack_workspace(c, S, L), lib.muon_workspace(mats)
    loss, lse = torch.empty(S, device="cuda"), torch.empty(S, device="cuda")
    d_hidden, d_stack = torch.empty_like(th), torch.empty_like(th)
    sumsq = torch.zeros(2, dtype=torch.float64, device="cuda")
    lists = [[d[k] for d in devs] for k in ("w", "a", "lq", "lv")]

    def step():
        lib.xent_forward(th, tw, tt, loss, lse, ws=ws_x)
        lib.xent_backward(th, tw, tt, lse, td, d_hidden, ws=ws_x)
        lib.rmsnorm_backward(tx, tg, d_hidden, eps, out=d_stack)
        lib.stack_backward(c, S, L, *lists, adam, d_stack, sumsq, ws_s)
        lib.muon(mats, mcfg, ws_m)

    step()
    for ws in (ws_x, ws_s, ws_m):
        lib.workspace_status(ws)
    after = [p.clone() for p in params]

    tol = (1e-5, 1e-4) if kind == "tiny" else (BF16_REL_L2, None)
    rloss, rlse = ops.xent_forward(hidden, host(tw), targets)
    check("loss", host(loss), rloss)
    rdh, _ = ops.xent_backward(hidden, host(tw), targets, rlse, d_loss)
    check("d_hidden", host(d_hidden), rdh)                     # float32 hidden rows: the float32 bar for both heads
    ref = OL.stack_backward(cfg, layers, ops.rmsnorm_backward(x, gamma, rdh, eps))
    check("d_in", host(d_stack), ref["d_in"], *tol)
    for l in range(n):
        for j, k in enumerate(names):
            i = l * len(names) + j
            check("layer %d %s" % (l, k), host(grads[i]), ref["layers"][l]["d" + k[0].upper() + k[1:]], *tol)
            g, p0 = host(grads[i]), host(before[i])
            rows, cols = p0.shape
            # the first step from zero momentum: u = g + mu g, and its direction is g's
            direction = ops.newton_schulz(g / np.linalg.norm(g), COEF, 5)
            move = 0.02 * np.sqrt(max(1.0, rows / cols))
            got = (p0 * (1 - 0.02 * 0.01) - host(after[i])) / move
            # p's own rounding, 2^-24 |p| twice, beside the update's bound
            limit = UPDATE_REL * np.linalg.norm(direction) + 2.0 ** -23 * np.linalg.norm(p0) / move
            assert np.linalg.norm(got - direction) <= limit, (l, k, np.linalg.norm(got - direction), limit)

    # the same step as one captured graph, from the same start
    for p, b, m in zip(params, before, momenta):
        p.copy_(b)
        m.zero_()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    graph.replay()
    torch.cuda.synchronize()
    for p, a in zip(params, after):
        assert torch.equal(p, a)
