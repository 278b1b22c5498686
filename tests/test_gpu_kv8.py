"""The 8-bit K/V cache on the GPU: rows as the float64 oracle quantises them, bit for bit, read back, and
attended by single tokens, with the gradient.

Tolerances of the attention: the stated float32 bar (relative L2 1e-5) for float32, half a bf16 step
(2^-8 of each value) more for bf16 results.
"""
import numpy as np
import pytest

from oracle import blocks8
from tests.helpers import F32_REL_L2, check, host

pytestmark = pytest.mark.gpu


def dev(x, bf16=False):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.bfloat16() if bf16 else t


def rows_of(n, heads, hd, seed=0):
    r = np.random.default_rng(seed)
    return (r.normal(size=(n, heads, hd)) * np.exp(r.normal(0, 1, (n, heads, 1)))).astype(np.float32)


def quantized(x):
    """(values [n, heads, hd], scales [heads, n]) of the oracle, one block a row and head."""
    n, heads, hd = x.shape
    v, s = blocks8.quantize(host(x).reshape(n * heads, hd), 1, hd)
    return v.reshape(x.shape), s.reshape(n, heads).T


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("hd", [16, 64, 96, 128, 256])
@pytest.mark.parametrize("rows,heads", [(1, 1), (7, 3), (200, 8)])
def test_write_and_read(lib, rows, heads, hd, bf16):
    import torch
    slots = np.random.default_rng(0).permutation(rows + 9)[:rows].astype(np.int64)
    if rows > 2:
        slots[1], slots[2] = -1, rows + 9                      # padding, and past the end
    cache = lib.kv8_cache(rows + 9, heads, hd)
    for t in cache.tensors:
        t.view(torch.uint8).fill_(0x11)
    before = [t.clone() for t in cache.tensors]
    k, v = dev(rows_of(rows, heads, hd, 1), bf16), dev(rows_of(rows, heads, hd, 2), bf16)
    lib.kv8_write(cache, k, v, dev(slots))
    used = (slots >= 0) & (slots < rows + 9)
    rest = np.setdiff1d(np.arange(rows + 9), slots[used])
    for x, codes, scales, b_codes, b_scales in ((k, *cache.tensors[:2], *before[:2]), (v, *cache.tensors[2:], *before[2:])):
        want, want_s = quantized(x)
        assert np.array_equal(host(codes.float())[slots[used]], want[used])
        assert np.array_equal(host(scales)[:, slots[used]], want_s[:, used])
        assert np.array_equal(host(codes.float())[rest], host(b_codes.float())[rest])     # other slots as they were
        assert np.array_equal(host(scales)[:, rest], host(b_scales)[:, rest])
    for dtype in (torch.float32, torch.bfloat16):
        for layout in ("shd", "hsd"):
            gk, gv = lib.kv8_read(cache, dev(slots), dtype, layout)
            for got, x in ((gk, k), (gv, v)):
                want, want_s = quantized(x)
                want = want * want_s.T[:, :, None]
                want[~used] = 0
                got = host(got).transpose(1, 0, 2) if layout == "hsd" else host(got)
                assert np.array_equal(got, want)               # 4 bits times a power of two: exact in both types


def test_read_of_any_scale(lib):
    import torch
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(2, 1, 128).view(torch.float8_e4m3fn)
    scales = torch.tensor([[0.3, 1.7e-3]], device="cuda")
    cache = lib.kv8_cache_of(codes, scales, codes.clone(), scales.clone())
    k, v = lib.kv8_read(cache, torch.tensor([1, 0, 1], device="cuda"))
    want = (codes.float() * scales.T[:, :, None])[[1, 0, 1]]
    assert torch.equal(k.nan_to_num(), want.nan_to_num()) and torch.equal(k.isnan(), want.isnan()) and torch.equal(v.nan_to_num(), k.nan_to_num())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
def test_write_from_a_fused_projection(lib, hd, bf16):
    """k and v as parts of one [rows, (2 + 2 + 2) heads of hd] tensor that starts anywhere."""
    import torch
    rows, heads = 21, 2
    for start in (0, 1):
        flat = dev(rows_of(1, 1, rows * 3 * heads * hd + start, 3)[0, 0], bf16)[start:]
        qkv = flat.reshape(rows, 3 * heads, hd)
        k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
        cache, other = lib.kv8_cache(rows, heads, hd), lib.kv8_cache(rows, heads, hd)
        slots = torch.arange(rows, device="cuda")
        lib.kv8_write(cache, k, v, slots)
        lib.kv8_write(other, k.contiguous(), v.contiguous(), slots)
        # heads ahead of positions, as a transposed tensor has them
        third = lib.kv8_cache(rows, heads, hd)
        lib.kv8_write(third, k.transpose(0, 1).contiguous().transpose(0, 1), v, slots)
        for t in (other, third):
            for a, b in zip(cache.tensors, t.tensors):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_values_that_are_not_finite_stay_in_their_row(lib):
    import torch
    x = rows_of(4, 2, 64)
    x[1, 0, 5], x[2, 1, 63] = np.nan, np.inf
    x[3] = 0
    cache = lib.kv8_cache(4, 2, 64)
    slots = torch.arange(4, device="cuda")
    lib.kv8_write(cache, dev(x), dev(x), slots)
    k, _ = lib.kv8_read(cache, slots)
    bad = torch.zeros(4, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    assert torch.equal(k.isnan(), bad[:, :, None].expand_as(k)) and torch.equal(k[3], torch.zeros(2, 64, device="cuda"))


# ---------------------------------------------------------------- attention

def problem(lib, lengths, heads, kv, hd, page, bf16=False, seed=0, longest=None, extra=3, poison=True, scales="any"):
    """A cache whose unused slots hold NaN codes and scales (what must not be looked at), pages in no order."""
    import torch
    r = np.random.default_rng(seed)
    n_seq, longest = len(lengths), max([1, *lengths]) if longest is None else longest
    most = -(-longest // page)
    n_pages = n_seq * most + extra
    pages = r.permutation(n_pages)[: n_seq * most].reshape(n_seq, most).astype(np.int32)
    cache = lib.kv8_cache(n_pages * page, kv, hd)
    if poison:
        for t in cache.tensors:
            t.view(torch.uint8).fill_(0xFF)
    K, V = [], []
    for b, n in enumerate(lengths):
        j = np.arange(n)
        slots = pages[b][j // page].astype(np.int64) * page + j % page
        k, v = rows_of(n, kv, hd, seed + 10 + b), rows_of(n, kv, hd, seed + 90 + b)
        if n:
            lib.kv8_write(cache, dev(k), dev(v), dev(slots))
            if scales == "any":                                # as another program may have chosen them
                f = dev(r.uniform(0.5, 1.0, (kv, n)).astype(np.float32))
                cache.tensors[1][:, dev(slots)] *= f
                cache.tensors[3][:, dev(slots)] *= f.flip(0)
        got = lib.kv8_read(cache, dev(slots))
        K.append(host(got[0]))
        V.append(host(got[1]))
    if n_seq > 1:
        pages[1, -(-lengths[1] // page):] = -1                 # pages past the last key are not looked at
    q = dev(r.normal(size=(n_seq, heads, hd)).astype(np.float32), bf16)
    g = dev((r.normal(size=(n_seq, heads, hd)) * 0.3).astype(np.float32), bf16)
    return cache, q, g, dev(pages), dev(np.array(lengths, np.int32)), longest, K, V


def cancelled(q, K, V, g, scale):
    """What d_q and d_k may be off by beside their own size, ds being a difference: dp_j and D = sum p dp are sums of
    head_dim products in float32, off by (head_dim + 8) 2^-24 of the sums of magnitudes m_j and sum p m, and p by
    4 |lse| 2^-24 of itself (s and lse are rounded where they are large), the same for all keys, which D feels and
    dp does not.  So ds_j is off by e p_j (m_j + sum p m), e = (head_dim + 8 + 4 |lse|) 2^-24, and d_q by scale times
    the sum of that and |k_j|."""
    n = len(K)
    group = q.shape[0] // K.shape[1]
    d_q, d_k = np.zeros_like(q), np.zeros(K.shape[1:])
    norms = blocks8.attention(q, K, V, scale)[1]
    for h in range(q.shape[0] if n else 0):
        lse = norms[h]
        p = np.exp(scale * K[:, h // group] @ q[h] - lse)
        m = np.abs(V[:, h // group]) @ np.abs(g[h])
        e = (q.shape[1] + 8 + 4 * abs(lse)) * 2.0 ** -24 * p * (m + p @ m) * abs(scale)
        d_q[h] = e @ np.abs(K[:, h // group])
        d_k[h // group] += e[-1] * np.abs(q[h])
    return d_q, d_k


def compare(name, got, want, bf16, more=(), rel=F32_REL_L2):
    got, want = host(got), np.stack(want)
    assert np.all(np.isfinite(got)), name
    norm = np.linalg.norm(want)
    off = np.linalg.norm(got - want)
    limit = (rel + (2.0 ** -8 if bf16 else 0)) * norm + 1e-30 + np.linalg.norm(np.stack(more) if len(more) else 0.0)
    assert off <= limit, "%s: %.3e of %.3e" % (name, off, norm)


def run(lib, lengths, heads, kv, hd, page, bf16=False, seed=0, scale=None, ws=True, **kw):
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, lengths, heads, kv, hd, page, bf16, seed, **kw)
    w = lib.kv8_attn_workspace(cache, len(lengths), heads, longest, grad=True) if ws else None
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, page, lens, longest, scale, ws=w)
    d_q, d_k, d_v = lib.kv8_attn_backward(cache, q, pages, page, lens, longest, lse, g, scale, ws=w)
    lib.workspace_status(w)
    at = hd ** -0.5 if scale is None else scale
    want = [blocks8.attention(host(q)[b], K[b], V[b], at) for b in range(len(lengths))]
    back = [blocks8.attention_backward(host(q)[b], K[b], V[b], host(g)[b], at) for b in range(len(lengths))]
    compare("ctx", ctx, [w_[0] for w_ in want], bf16)
    rlse = np.stack([w_[1] for w_ in want])
    empty = np.isinf(rlse)
    assert np.array_equal(np.isinf(host(lse)), empty) and np.all(host(lse)[empty] < 0)
    # logits of magnitude m carry m 2^-22 or so, and lse lies within log(n) of the largest
    assert np.max(np.abs(host(lse)[~empty] - rlse[~empty]) / np.maximum(1, np.abs(rlse[~empty])), initial=0) <= 1e-5
    more = [cancelled(host(q)[b], K[b], V[b], host(g)[b], at) for b in range(len(lengths))]
    for name, got, i in (("d_q", d_q, 0), ("d_k", d_k, 1), ("d_v", d_v, 2)):
        compare(name, got, [b_[i] for b_ in back], bf16, [m[i] for m in more] if i < 2 else ())
    again = lib.kv8_attn_forward(cache, q, pages, page, lens, longest, scale, ws=w)
    assert torch.equal(ctx, again[0]) and torch.equal(lse, again[1])
    again = lib.kv8_attn_backward(cache, q, pages, page, lens, longest, lse, g, scale, ws=w)
    assert all(torch.equal(a, b) for a, b in zip((d_q, d_k, d_v), again))


CASES = [([1], 1, 1, 16, 1), ([1, 0, 2], 4, 2, 64, 16), ([5, 16, 17], 3, 1, 64, 4), ([33, 64, 100, 7], 8, 8, 128, 64),
         ([1024], 20, 5, 128, 64), ([300, 31, 1], 32, 8, 128, 16), ([129], 8, 1, 96, 100), ([77, 128], 16, 1, 128, 7),
         ([40, 41], 12, 1, 256, 32), ([700, 3, 250, 0, 1], 4, 1, 256, 64), ([513], 5, 5, 32, 1), ([2000, 1500], 24, 8, 64, 64),
         ([90], 9, 3, 48, 33), ([0], 4, 4, 64, 8), ([18], 33, 1, 112, 5)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("lengths,heads,kv,hd,page", CASES)
def test_attention(lib, lengths, heads, kv, hd, page, bf16):
    run(lib, lengths, heads, kv, hd, page, bf16, seed=len(lengths) + hd)


def test_one_key_has_no_gradient(lib):
    """Of a sequence of one key d_q and d_k are 0 exactly, and its value's gradient is d_ctx summed over the heads."""
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [1, 1, 40], 8, 2, 64, 16, seed=8)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    d_q, d_k, d_v = lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g)
    assert torch.count_nonzero(d_q[:2]) == 0 and torch.count_nonzero(d_k[:2]) == 0 and torch.count_nonzero(d_q[2]) > 0
    compare("d_v", d_v[:2], list(host(g)[:2].reshape(2, 2, 4, 64).sum(2)), False)


def test_attention_of_a_long_sequence(lib):
    run(lib, [20011], 8, 2, 128, 64, seed=3)


def test_attention_of_many_sequences(lib):
    run(lib, [int(x) for x in np.random.default_rng(1).integers(0, 90, 150)], 8, 2, 64, 16, seed=4)


def test_attention_with_a_workspace_of_its_own_and_another_scale(lib):
    run(lib, [300, 20], 8, 2, 128, 64, seed=5, scale=0.5, ws=None)


@pytest.mark.parametrize("scale", [0.0, 3.0, -1.0])
def test_attention_flat_and_sharp(lib, scale):
    """All weights equal, one near 1 (the bar holds in the norm), and a scale below 0."""
    run(lib, [400, 60], 8, 2, 64, 16, seed=6, scale=scale)


def test_lengths_beyond_max_len_and_the_pages(lib):
    """A length past max_len or the pages counts as the smaller one."""
    import torch
    cache, q, g, pages, lens, _, K, V = problem(lib, [64], 4, 2, 64, 16)
    for most, n in ((40, 40), (1 << 20, 64)):
        ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, torch.tensor([1 << 30], dtype=torch.int32, device="cuda"), most)
        want = blocks8.attention(host(q)[0], K[0][:n], V[0][:n], 0.125)
        compare("ctx", ctx, [want[0]], False)
        compare("lse", lse, [want[1]], False)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, torch.tensor([-5], dtype=torch.int32, device="cuda"), 64)
    assert torch.all(ctx == 0) and torch.all(lse == -float("inf"))


def test_pages_that_are_not_there(lib):
    """Keys on a page outside the cache are left out; where none is left the row is empty."""
    import torch
    cache, q, g, pages, lens, _, K, V = problem(lib, [100, 30], 8, 2, 64, 16)
    pages[0, 2], pages[0, 4] = -1, 1 << 30
    pages[1] = -7
    kept = np.r_[0:32, 48:64, 80:100]
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, 100)
    want = blocks8.attention(host(q)[0], K[0][kept], V[0][kept], 0.125)
    compare("ctx", ctx[0], [want[0]], False)
    assert torch.all(ctx[1] == 0) and torch.all(lse[1] == -float("inf"))
    d_q, d_k, d_v = lib.kv8_attn_backward(cache, q, pages, 16, lens, 100, lse, g)
    back = blocks8.attention_backward(host(q)[0], K[0][kept], V[0][kept], host(g)[0], 0.125)
    for got, w in ((d_q, back[0]), (d_k, back[1]), (d_v, back[2])):
        compare("gradient", got[0], [w], False)
        assert torch.all(got[1] == 0)
    # the newest key's page missing: no gradient of it
    pages[0, 6] = -1
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, 100)
    d_q, d_k, d_v = lib.kv8_attn_backward(cache, q, pages, 16, lens, 100, lse, g)
    assert torch.all(d_k[0] == 0) and torch.all(d_v[0] == 0) and torch.all(d_q[0].isfinite())
    none = lib.kv8_attn_forward(cache, q, pages[:, :0], 16, lens, 100)
    assert torch.all(none[0] == 0) and torch.all(none[1] == -float("inf"))


def test_a_page_shared_by_sequences(lib):
    """Sequences may share pages (a common prompt)."""
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [64], 4, 2, 64, 16)
    two = q.repeat(3, 1, 1)
    ctx, lse = lib.kv8_attn_forward(cache, two, pages.repeat(3, 1), 16, torch.tensor([64, 17, 64], dtype=torch.int32, device="cuda"), 64)
    one = lib.kv8_attn_forward(cache, q, pages, 16, lens, 64)
    short = blocks8.attention(host(q)[0], K[0][:17], V[0][:17], 0.125)
    assert torch.equal(ctx[0], ctx[2])
    compare("ctx", ctx[0], [host(one[0])[0]], False)
    compare("ctx", ctx[1], [short[0]], False)


def test_weights_of_very_different_size(lib):
    """One key that takes nearly all the weight beside many that share the rest, and values whose scales differ
    by 2^20: what is small by itself still adds up."""
    import torch
    n, hd = 4000, 64
    r = np.random.default_rng(2)
    k, v = rows_of(n, 1, hd, 1) * 0.01, r.uniform(0.9, 1.0, (n, 1, hd)).astype(np.float32)
    k[7] = 3.0
    v[7] *= np.float32(2.0 ** -20)
    v[9] *= np.float32(2.0 ** 10)
    cache = lib.kv8_cache(n, 1, hd)
    slots = torch.arange(n, device="cuda")
    lib.kv8_write(cache, dev(k), dev(v), slots)
    K, V = (host(t) for t in lib.kv8_read(cache, slots))
    q = dev(np.full((1, 2, hd), 0.9, np.float32))
    g = dev(np.random.default_rng(3).normal(size=(1, 2, hd)).astype(np.float32))
    args = (cache, q, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), n, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    ctx, lse = lib.kv8_attn_forward(*args, scale=0.1)
    # the logit of the large key, a sum of 64 products, is off by up to 68 x 2^-24 of the sum of magnitudes (17.3),
    # and the weight of every other key by that much of itself: 7.0e-5
    rel = F32_REL_L2 + 68 * 2.0 ** -24 * 0.1 * float(np.max(np.abs(K[:, 0]) @ np.abs(host(q)[0, 0])))
    want, back = blocks8.attention(host(q)[0], K, V, 0.1), blocks8.attention_backward(host(q)[0], K, V, host(g)[0], 0.1)
    compare("ctx", ctx, [want[0]], False, rel=rel)
    compare("lse", lse, [want[1]], False)
    d_q, d_k, d_v = lib.kv8_attn_backward(*args, lse, g, scale=0.1)
    more = cancelled(host(q)[0], K, V, host(g)[0], 0.1)
    compare("d_q", d_q, [back[0]], False, [more[0]], rel)
    compare("d_k", d_k, [back[1]], False, [more[1]], rel)
    compare("d_v", d_v, [back[2]], False, rel=rel)


@pytest.mark.parametrize("power", [-110, 110, 118])
def test_values_of_extreme_scales(lib, power):
    """Values whose scales are near the ends of float32: results are those of ordinary ones times the power."""
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [150, 20], 8, 2, 64, 16, seed=11)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    cache.tensors[3].mul_(2.0 ** power)
    far, lse2 = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    assert torch.equal(lse, lse2) and torch.all(far.isfinite())
    # products with a power of two are exact; sums are held to the same number of bits at any of them
    check("ctx", host(far * 2.0 ** -power), host(ctx), rel_l2=2 * F32_REL_L2, max_abs=None)


def test_only_the_status_block_is_cleared(lib):
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [900, 33, 0], 8, 2, 128, 16)
    got = []
    for fill in (0, 255):
        ws = lib.kv8_attn_workspace(cache, 3, 8, longest, grad=True)
        ws[256:] = fill
        ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest, ws=ws)
        ws[256:] = fill
        got.append((ctx, lse, *lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g, ws=ws)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    with pytest.raises(lib.TlbError, match="workspace"):
        lib.kv8_attn_forward(cache, q, pages, 16, lens, longest, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
