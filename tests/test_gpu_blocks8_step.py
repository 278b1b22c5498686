"""The 8-bit operators as they are used together: a token's key and value into the cache, attention over it, its
gradient, back through the rotary embedding and the frozen 8-bit projection; eager, on another stream and as
captured graphs, against the float64 oracle and against the layer calls on the cache read back.

Tolerances: float32 paths at the stated bar (relative L2 1e-5).  The 8-bit product is compared with the oracle's on
the same quantised operands.
"""
import numpy as np
import pytest

from oracle import blocks8, ops
from tests.helpers import F32_MAX_ABS, F32_REL_L2, check, host
from tests.test_gpu_fp8 import operands
from tests.test_gpu_kv8 import dev, problem, rows_of

pytestmark = pytest.mark.gpu


class Token:
    """One token of a sequence of n keys: 8 query heads over 2 KV heads of 64, a hidden size of 384."""
    n, heads, kv, hd, dim, page = 333, 8, 2, 64, 384, 16

    def __init__(self, lib, seed=0):
        import torch
        r = np.random.default_rng(seed)
        self.lib = lib
        self.cache, self.q, self.g, self.pages, self.lens, self.longest, self.K, self.V = problem(
            lib, [self.n], self.heads, self.kv, self.hd, self.page, seed=seed, scales="powers")
        self.k, self.v = dev(rows_of(1, self.kv, self.hd, seed + 5)), dev(rows_of(1, self.kv, self.hd, seed + 6))
        j = self.n - 1
        slot = int(self.pages[0, j // self.page]) * self.page + j % self.page
        self.slots = torch.tensor([slot], device="cuda")
        self.W, self.w_s = lib.fp8_quantize(dev((r.normal(size=(self.dim, self.heads * self.hd)) * 0.05).astype(np.float32)), 128)
        self.ws = lib.kv8_attn_workspace(self.cache, 1, self.heads, self.longest, grad=True)
        self.ws_l = lib.linear_fp8_workspace(1, self.heads * self.hd, self.dim)
        self.d_n1 = torch.zeros(1, self.dim, device="cuda")

    def step(self, stream=None):
        lib = self.lib
        lib.kv8_write(self.cache, self.k, self.v, self.slots, stream=stream)
        over = (self.cache, self.q, self.pages, self.page, self.lens, self.longest)
        ctx, lse = lib.kv8_attn_forward(*over, ws=self.ws, stream=stream)
        d_q, d_k, d_v = lib.kv8_attn_backward(*over, lse, self.g, ws=self.ws, stream=stream)
        d_qpre = lib.rope_backward(d_q, self.n - 1, stream=stream)
        codes, scales = lib.fp8_quantize(d_qpre.reshape(1, -1), stream=stream)
        lib.linear_fp8_backward(self.W, self.w_s, codes, scales, out=self.d_n1, ws=self.ws_l, stream=stream)
        return ctx, lse, d_q, d_k, d_v, d_qpre, codes, scales

    def expected(self):
        values, scales = blocks8.quantize(host(self.k).reshape(self.kv, self.hd), 1, self.hd)
        K, V = self.K[0].copy(), self.V[0].copy()
        K[-1] = values * scales
        values, scales = blocks8.quantize(host(self.v).reshape(self.kv, self.hd), 1, self.hd)
        V[-1] = values * scales
        q, g, at = host(self.q)[0], host(self.g)[0], self.hd ** -0.5
        return blocks8.attention(q, K, V, at) + blocks8.attention_backward(q, K, V, g, at), K, V


def test_a_token_through_the_cache_and_the_projection(lib):
    import torch
    t = Token(lib)
    ctx, lse, d_q, d_k, d_v, d_qpre, codes, scales = t.step()
    lib.workspace_status(t.ws_l)
    (rctx, rlse, rq, rk, rv), K, V = t.expected()
    for name, got, want in (("ctx", ctx[0], rctx), ("lse", lse[0], rlse), ("d_q", d_q[0], rq), ("d_k", d_k[0], rk), ("d_v", d_v[0], rv)):
        check(name, host(got), want)
    check("d_qpre", host(d_qpre[0]), ops.rope_backward(rq[None], t.n - 1, 10000.0)[0])
    check("d_n1", host(t.d_n1), blocks8.linear_backward(host(t.W.float()), host(t.w_s), host(codes.float()), host(scales)))
    # the same step on a stream of its own, and as two captured graphs replayed in turn
    first = [x.clone() for x in (ctx, lse, d_q, d_k, d_v, t.d_n1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t.d_n1.zero_()
    side.wait_stream(torch.cuda.current_stream())
    again = t.step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again[:5] + (t.d_n1,)))
    other = Token(lib, seed=30)
    want = [x.clone() for x in other.step()[:5]] + [other.d_n1.clone()]
    graphs = []
    for token in (t, other):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            outs = token.step()
        graphs.append((graph, outs))
    for _ in range(3):
        for token, (graph, _) in zip((t, other), graphs):
            token.d_n1.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for token, outs, ref in ((t, graphs[0][1], first), (other, graphs[1][1], want)):
        assert all(torch.equal(a, b) for a, b in zip(outs[:5] + (token.d_n1,), ref))


def test_gradient_is_the_layer_calls_on_the_cache_read_back(lib):
    """tlb_attn_backward with recomputed weights, on the keys and values that kv8_read gives and the lse that the
    forward gave, finds the same gradients (an identity for the O projection hands it d_ctx)."""
    import torch
    t = Token(lib, seed=7)
    ctx, lse, d_q, d_k, d_v, d_qpre, _, _ = t.step()
    j = torch.arange(t.n, device="cuda")
    slots = t.pages[0].long()[j // t.page] * t.page + j % t.page
    for layout in ("shd", "hsd"):
        k, v = lib.kv8_read(t.cache, slots, kv_layout=layout)
        dim = t.heads * t.hd
        c = lib.layer_cfg(dim, 64, t.heads, t.kv, t.hd, 4, 8.0, residual=False, rope=True, recompute_p=True)
        weights = {"w_o": torch.eye(dim, device="cuda")}
        weights.update({n: torch.zeros(64, dim, device="cuda") for n in ("w_down",)})
        weights.update({n: torch.zeros(dim, 64, device="cuda") for n in ("w_gate", "w_up")})
        w = lib.layer_weights(c, weights)
        acts = {"k": k, "v": v, "q": t.q.reshape(1, dim), "lse": lse.reshape(t.heads, 1)}
        a = lib.layer_acts(c, acts, layout, t.n)
        out_q, out_v = torch.empty(1, dim, device="cuda"), torch.empty(1, t.kv * t.hd, device="cuda")
        ws = lib.workspace(c, 1, t.n)
        lib.attn_backward(c, 1, t.n, t.g.reshape(1, dim), w, a, out_q, out_v, ws)
        lib.workspace_status(ws)
        # each is within the bar of the exact gradient, so they are within twice the bar of one another
        check("d_qpre", host(d_qpre).ravel(), host(out_q).ravel(), rel_l2=2 * F32_REL_L2, max_abs=2 * F32_MAX_ABS)
        check("d_v", host(d_v).ravel(), host(out_v).ravel(), rel_l2=2 * F32_REL_L2, max_abs=2 * F32_MAX_ABS)


def test_sequence_cached_in_8_bits_and_its_gradient_through_8_bit_weights(lib):
    """A sequence's keys and values written at once and read back for a layer call, and a sequence's gradient through a
    frozen weight held in 8 bits: the few-rows and the tensor-core product agree on the rows they share."""
    import torch
    S, out, dim = 100, 384, 256
    W, w_s = lib.fp8_quantize(dev((np.random.default_rng(1).normal(size=(dim, out)) * 0.05).astype(np.float32)), 128)
    g = dev(rows_of(S, 3, 128, 4).reshape(S, out))
    q, s = lib.fp8_quantize(g)
    first = lib.launch_count()
    all_rows = lib.linear_fp8_backward(W, w_s, q, s)
    few = lib.linear_fp8_backward(W, w_s, q[:7], s[:7])
    names = lib.launch_names(first)
    assert "linear_fp8_tc" in names and "linear_fp8_rows" in names
    ref = blocks8.linear_backward(host(W.float()), host(w_s), host(q.float()), host(s))
    check("all rows", host(all_rows), ref)
    check("few rows", host(few), ref[:7])
    lib.workspace_status()
    k, v = dev(rows_of(S, 2, 64, 8)), dev(rows_of(S, 2, 64, 9))
    cache = lib.kv8_cache(S, 2, 64)
    slots = torch.arange(S, device="cuda")
    lib.kv8_write(cache, k, v, slots)
    bk, bv = lib.kv8_read(cache, slots)
    for got, x in ((bk, k), (bv, v)):
        # half a step of three bits after the leading one, or of the smallest step: 2^-10 of the row's scale, which is
        # at most 2^-8 of its largest value's power of two
        top = x.abs().amax(2, keepdim=True)
        assert torch.all((got - x).abs() <= torch.maximum(x.abs() * 2.0 ** -4, top * 2.0 ** -17))


@pytest.mark.parametrize("S", [1, 20, 200])
def test_linear_on_another_stream_while_the_current_one_works(lib, S):
    """Operands made on one stream and used on another that waits for it."""
    import torch
    W, w_s, dY, y_s = operands(S, 640, 512, 3)
    want = lib.linear_fp8_backward(W, w_s, dY, y_s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.linear_fp8_backward(W, w_s, dY, y_s, stream=side)
    with torch.cuda.stream(side):
        inside = lib.linear_fp8_backward(W, w_s, dY, y_s)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(inside, want)
    lib.workspace_status()
