"""How many bits the 8-bit operators keep on ordinary inputs, where a lost half of an operand (11 bits) would stay
below the bounds that hold for every input.

Roundings are taken as independent: a result's error is the root of the sum of its terms' squares, and the bar is
three times that.  u = 2^-23 is the most that one rounding of a sum (2^-24, or twice that where bits are cut off) or the
two halves of an operand are off by, relative to what is rounded.

Attention, of one query head, with a = sqrt(2 + head_dim / 16) (the two operands' halves, and a rounding for each 16 products):
  s_j   u a scale |q o k_j|  (o: value by value, | | the root of the squares' sum)  +  u |s_j|, twice: its two products
  p_j   p_j (that of s_j, + u for 2^x)         and all p alike: u (|lse| + 1), of lse
  dp_j  u a |d_ctx o v_j|
  D     the p_j dp_j's, each by p_j's and dp_j's, and u D sqrt(n / 64 + 8) for its sum
  sums over keys, of weights x_j: the terms' own errors, and u |sum| sqrt(n / 64 + 8), |sum| that of magnitudes
"""
import numpy as np
import pytest

from oracle import blocks8
from tests.helpers import host
from tests.test_gpu_fp8 import operands
from tests.test_gpu_kv8 import CASES, problem

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def norm(x, axis=None):
    return np.sqrt(np.sum(np.square(x), axis=axis))


def expected_errors(q, K, V, g, scale):
    """Root mean square errors (norms over each result) of ctx, d_q, d_k and d_v of one sequence."""
    n, kv, hd = K.shape
    group, a, adds = q.shape[0] // kv, np.sqrt(2 + hd / 16), np.sqrt(n / 64 + 8)
    norms = blocks8.attention(q, K, V, scale)[1]
    e_ctx, e_dq, e_dk, e_dv = np.zeros(len(q)), np.zeros(len(q)), np.zeros(kv), np.zeros(kv)
    for h in range(len(q)):
        k, v = K[:, h // group], V[:, h // group]
        s = scale * k @ q[h]
        p, dp = np.exp(s - norms[h]), v @ g[h]
        D, z = p @ dp, p @ k
        nk, nv, ctx = norm(k, 1), norm(v, 1), p @ v
        e_s = np.sqrt((U * a * abs(scale) * norm(k * q[h], 1)) ** 2 + 2 * (U * s) ** 2)
        e_p = p * np.sqrt(e_s ** 2 + U ** 2)
        e_dp = U * a * norm(v * g[h], 1)
        all_p = U * (abs(norms[h]) + 1)
        e_D = norm(np.concatenate([e_p * dp, p * e_dp, [U * adds * (p @ np.abs(dp))]]))
        e_ctx[h] = norm(np.concatenate([e_p * norm(v - ctx, 1), [U * adds * norm(p @ np.abs(v))]]))
        e_dq[h] = abs(scale) * norm(np.concatenate([
            e_p * norm(k * (dp - D)[:, None] - D * z, 1) if n > 1 else [0.0],
            p * e_dp * nk, p * np.abs(dp) * nk * U, [e_D * norm(z), all_p * norm(D * z)],
            [U * adds * norm((p * np.abs(dp)) @ np.abs(k)), U * adds * abs(D) * norm(p @ np.abs(k))]]))
        last = abs(p[-1]) * norm([e_dp[-1], e_D, abs(dp[-1] - D) * (e_p[-1] / p[-1] + all_p + U), abs(D) * all_p])
        e_dk[h // group] = norm([e_dk[h // group], abs(scale) * last * norm(q[h])])
        e_dv[h // group] = norm([e_dv[h // group], norm([e_p[-1], p[-1] * all_p, p[-1] * U]) * norm(g[h])])
    return norm(e_ctx), norm(e_dq), norm(e_dk), norm(e_dv)


def held(name, got, want, errors):
    off, limit = norm(host(got) - np.stack(want)), 3 * norm(errors) + 1e-30
    print("%s: %.2e of %.2e, bar %.2e" % (name, off, norm(want), limit))
    assert off <= limit, "%s: off by %.3e, at most %.3e (its norm %.3e)" % (name, off, limit, norm(want))


def attention(lib, lengths, heads, kv, hd, page, seed, flat=1.0):
    cache, q, g, pages, lens, longest, K, V = problem(lib, lengths, heads, kv, hd, page, seed=seed)
    Q, G, scale = host(q), host(g), float(np.float32(flat * hd ** -0.5))
    w = lib.kv8_attn_workspace(cache, len(lengths), heads, longest, grad=True)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, page, lens, longest, scale, ws=w)
    grads = lib.kv8_attn_backward(cache, q, pages, page, lens, longest, lse, g, scale, ws=w)
    want = [(blocks8.attention(Q[b], K[b], V[b], scale)[0], *blocks8.attention_backward(Q[b], K[b], V[b], G[b], scale))
            for b in range(len(lengths))]
    errors = np.array([expected_errors(Q[b], K[b], V[b], G[b], scale) for b in range(len(lengths)) if lengths[b]]).reshape(-1, 4)
    for i, (name, got) in enumerate(zip(("ctx", "d_q", "d_k", "d_v"), (ctx, *grads))):
        held(name, got, [w_[i] for w_ in want], errors[:, i])


# Logits spread as they are, and closer together: the fewer keys share the weight, the more of d_q cancels and the wider
# its bar.  With 0.3 (ctx) and 0.1 (gradients) of the scale operands of 11 bits miss the bars 5 to 200 times over.
FLAT = [1.0, 0.3, 0.1]


@pytest.mark.parametrize("flat", FLAT)
@pytest.mark.parametrize("lengths,heads,kv,hd,page", CASES)
def test_attention(lib, lengths, heads, kv, hd, page, flat):
    attention(lib, lengths, heads, kv, hd, page, len(lengths) + hd, flat)


@pytest.mark.parametrize("flat", FLAT)
def test_attention_in_many_parts(lib, flat):
    attention(lib, [20011], 8, 2, 128, 64, 3, flat)


@pytest.mark.parametrize("flat", FLAT)
def test_attention_of_many_sequences(lib, flat):
    attention(lib, [int(x) for x in np.random.default_rng(1).integers(0, 90, 150)], 8, 2, 64, 16, 4, flat)


@pytest.mark.parametrize("S,out,dim", [(1, 9728, 2560), (8, 4096, 512), (9, 384, 640), (64, 2560, 2560), (200, 3000, 515),
                                       (333, 1001, 4099), (1030, 656, 1300)])
def test_linear(lib, S, out, dim):
    """The sum over a block of 128 columns is off by 2 u of itself (its products are exact, their sum is float32: a few
    roundings of the tensor core's), the product of the scales by u and the sum over blocks by u a block."""
    import torch
    W, w_s, dY, y_s = operands(S, out, dim, seed=S)
    got = lib.linear_fp8_backward(W, w_s, dY, y_s)
    lib.workspace_status()
    ref = blocks8.linear_backward(host(W.float()), host(w_s), host(dY.float()), host(y_s))
    held("dX", got, ref, U * norm(ref) * np.sqrt(5 + w_s.shape[1]))


@pytest.mark.parametrize("power", [-110, -60, 60, 110, 118])
def test_gradient_at_extreme_value_scales(lib, power):
    """Values near the ends of float32: d_v does not know, d_q and d_k are the ordinary ones times the power.  Products
    with a power of two are exact; each of the two is within the bar of its exact one."""
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [150, 20], 8, 2, 64, 16, seed=11)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    ordinary = lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g)
    cache.tensors[3].mul_(2.0 ** power)
    far = lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g)
    assert torch.equal(far[2], ordinary[2])
    errors = np.array([expected_errors(host(q)[b], K[b], V[b], host(g)[b], 0.125) for b in range(2)])
    for i in (0, 1):
        assert torch.all(far[i].isfinite())
        held("gradient", far[i].double() * 2.0 ** -power, host(ordinary[i]), 2 * errors[:, 1 + i])


@pytest.mark.parametrize("power", [-100, -60, 60, 100])
def test_attention_at_extreme_key_scales(lib, power):
    """Keys times 2^power and queries divided by it: the logits stay, and with them ctx and d_v; d_q grows and d_k falls."""
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [150, 20], 8, 2, 64, 16, seed=12)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    ordinary = lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g)
    cache.tensors[1].mul_(2.0 ** power)
    q2 = q * 2.0 ** -power
    ctx2, lse2 = lib.kv8_attn_forward(cache, q2, pages, 16, lens, longest)
    far = lib.kv8_attn_backward(cache, q2, pages, 16, lens, longest, lse2, g)
    errors = np.array([expected_errors(host(q)[b], K[b], V[b], host(g)[b], 0.125) for b in range(2)])
    held("ctx", ctx2, host(ctx), 2 * errors[:, 0])
    for i, shift in ((0, -power), (1, power), (2, 0)):
        assert torch.all(far[i].isfinite())
        held("gradient", far[i].double() * 2.0 ** shift, host(ordinary[i]), 2 * errors[:, 1 + i])
