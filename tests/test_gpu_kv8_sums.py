"""The sums of the 8-bit cache's attention where keys differ by many powers of two.

Tolerances: the stated float32 bar (relative L2 1e-5), and beside it what the size of the logits costs where they are
not all equal: s is a float32 (its product with the scale, and with log2 e, rounded once each, 4 |s| 2^-24 with the
sum's own roundings), and a weight is off by as much of itself as its logit is absolutely.
"""
import numpy as np
import pytest

from oracle import blocks8
from tests.helpers import F32_REL_L2, host
from tests.test_gpu_kv8 import cancelled, compare, dev

pytestmark = pytest.mark.gpu


def cache_of(lib, k, v, k_scale, v_scale):
    """A cache of these e4m3 values [n, heads, hd] and scales [n], the same for all heads."""
    import torch
    codes = [torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.float8_e4m3fn) for x in (k, v)]
    scales = [dev(np.tile(np.asarray(s, np.float32), (k.shape[1], 1))) for s in (k_scale, v_scale)]
    return lib.kv8_cache_of(codes[0], scales[0], codes[1], scales[1])


@pytest.mark.parametrize("spread", [0, 20, 30, 40, 100])
@pytest.mark.parametrize("gap", [40, 150])
def test_a_large_value_that_lost_its_weight(lib, gap, spread):
    """80 keys, five steps of one CTA: a value 2^spread the others' size among a warp's first 16 keys, and logits higher
    by gap in its second step.  The 16 keys that take the weight have one logit, so its rounding cancels."""
    import torch
    r = np.random.default_rng(spread)
    n, hd = 80, 64
    k = np.zeros((n, 1, hd), np.float32)
    k[64:] = 1.0
    v = r.integers(-15, 16, (n, 1, hd)).astype(np.float32)
    v_scale = r.uniform(0.5, 1.0, n).astype(np.float32)
    v_scale[3] = 2.0 ** spread
    cache = cache_of(lib, k, v, np.ones(n), v_scale)
    q = dev(np.full((1, 2, hd), 1.0, np.float32))
    args = (cache, q, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), n, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    K, V = k.astype(np.float64), v.astype(np.float64) * v_scale.astype(np.float64)[:, None, None]
    ctx, lse = lib.kv8_attn_forward(*args, scale=gap / hd)
    want = blocks8.attention(host(q)[0], K, V, float(np.float32(gap / hd)))
    # where the early value still counts (e^-40 2^100), its weight is off by 4 gap 2^-24 of itself
    compare("ctx", ctx, [want[0]], False, rel=F32_REL_L2 + (4 * gap * 2.0 ** -24 if spread * np.log(2) > gap - 12 else 0))
    compare("lse", lse, [want[1]], False)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("rise,fall", [(12, 12), (3, 4), (20, 16), (12, -8), (-6, 0)])
def test_logits_that_rise_while_values_shrink(lib, rise, fall, hd, bf16):
    """Ten steps of each warp (700 sequences of 640 keys on shared pages, a sequence a CTA or so): with each, logits
    rise by rise and values fall by 2^fall."""
    import torch
    r = np.random.default_rng(hd)
    n, seqs, page = 640, 700, 64
    step = np.arange(n) // 64
    k = np.broadcast_to((step if rise > 0 else 9 - step)[:, None, None], (n, 1, hd)).astype(np.float32)
    v = r.integers(-15, 16, (n, 1, hd)).astype(np.float32)
    v_scale = 2.0 ** (-fall * (step - 4.0))
    cache = cache_of(lib, k, v, np.ones(n), v_scale)
    # queries whose values sum to hd in a few bits: logits are step * |rise| * (1 or 7/8) up to their rounding
    factor = np.where(np.arange(seqs) % 2, 1.0, 0.875)
    q = dev(np.broadcast_to(factor[:, None, None], (seqs, 1, hd)).astype(np.float32), bf16)
    g = dev((r.integers(-8, 9, (1, 1, hd)) / 8).astype(np.float32).repeat(seqs, 0), bf16)
    pages = torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    scale = float(np.float32(abs(rise) / hd))
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, page, lens, n, scale)
    V = v.astype(np.float64) * v_scale[:, None, None]
    two = [blocks8.attention(host(q)[i], k.astype(np.float64), V, scale) for i in range(2)]
    most = 4 * 9 * abs(rise) * 2.0 ** -24
    for i in range(2):                                         # sequences of one query: the same bits, however they are shared out
        compare("ctx", ctx[i::2], [two[i][0]] * (seqs // 2), bf16, rel=F32_REL_L2 + most)
        compare("lse", lse[i::2], [two[i][1]] * (seqs // 2), False)
    d_q, d_k, d_v = lib.kv8_attn_backward(cache, q, pages, page, lens, n, lse, g, scale)
    back = [blocks8.attention_backward(host(q)[i], k.astype(np.float64), V, host(g)[i], scale) for i in range(2)]
    more = [cancelled(host(q)[i], k.astype(np.float64), V, host(g)[i], scale) for i in range(2)]
    for i in range(2):
        for name, got, w in (("d_q", d_q, 0), ("d_k", d_k, 1), ("d_v", d_v, 2)):
            compare(name, got[i::2], [back[i][w]] * (seqs // 2), bf16, [more[i][w]] * (seqs // 2) if w < 2 else (),
                    rel=F32_REL_L2 + most)
