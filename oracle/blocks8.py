"""8-bit blocks, the product of operands held that way, and single-token attention over an
8-bit K/V cache, in float64 numpy.

TEST INFRASTRUCTURE ONLY (see ``ops``).  e4m3 values are written out as a table of their 256
codes (sign, 4 exponent bits of bias 7, 3 mantissa bits; the two codes with all of these set are
NaN), and a value is rounded by looking for the nearest code.
"""
from __future__ import annotations

import numpy as np

from .ops import f64


def _value(code: int) -> float:
    sign, e, m = (-1.0 if code & 0x80 else 1.0), (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


E4M3 = np.array([_value(c) for c in range(256)])
_POSITIVE = E4M3[:127]                     # 0 .. 448, in order of their codes


def to_e4m3(x) -> np.ndarray:
    """The nearest e4m3 value of each |x| <= 448, of two equally near the one with an even code; NaN stays."""
    x = f64(x)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    below, above = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), np.nan, np.copysign(_POSITIVE[code], x))


def block_scale(block) -> float:
    """The smallest 2^e, e >= -126, with max|block| <= 448 * 2^e; NaN where the block is not finite."""
    block = f64(block)
    if not np.all(np.isfinite(block)):
        return float("nan")
    top, e = float(np.max(np.abs(block), initial=0.0)), -126
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def quantize(x, block_rows: int, block_cols: int = 128):
    """(values, scales) of x [rows, cols] in blocks of block_rows x block_cols."""
    x = f64(x)
    rows, cols = x.shape
    scales = np.zeros((-(-rows // block_rows), -(-cols // block_cols)))
    values = np.zeros_like(x)
    for r in range(scales.shape[0]):
        for c in range(scales.shape[1]):
            at = np.s_[r * block_rows:(r + 1) * block_rows, c * block_cols:(c + 1) * block_cols]
            scales[r, c] = s = block_scale(x[at])
            values[at] = to_e4m3(x[at] / s)
    return values, scales


def spread(scales, block_rows: int, rows: int, cols: int) -> np.ndarray:
    """The scale of every element of a [rows, cols] matrix."""
    return np.repeat(np.repeat(f64(scales), block_rows, 0)[:rows], 128, 1)[:, :cols]


def linear_backward(W, w_scales, dY, dy_scales) -> np.ndarray:
    """dX = dY W^T of the blocks' values: W [in, out], dY [S, out]."""
    w = f64(W) * spread(w_scales, 128, *np.shape(W))
    return (f64(dY) * spread(dy_scales, 1, *np.shape(dY))) @ w.T


def attention(q, K, V, scale: float):
    """(ctx, lse) of one query row a head: q [nh, hd], K and V [n, n_kv, hd]; head h reads h // (nh / n_kv)."""
    q, K, V = f64(q), f64(K), f64(V)
    group = q.shape[0] // K.shape[1]
    ctx, lse = np.zeros_like(q), np.full(q.shape[0], -np.inf)
    for h in range(q.shape[0] if len(K) else 0):
        s = scale * K[:, h // group] @ q[h]
        lse[h] = s.max() + np.log(np.sum(np.exp(s - s.max())))
        ctx[h] = np.exp(s - lse[h]) @ V[:, h // group]
    return ctx, lse


def attention_backward(q, K, V, d_ctx, scale: float):
    """(d_q, d_k, d_v): d_k and d_v [n_kv, hd] of the last key and value alone."""
    q, K, V, d_ctx = f64(q), f64(K), f64(V), f64(d_ctx)
    group = q.shape[0] // K.shape[1]
    d_q, d_k, d_v = np.zeros_like(q), np.zeros(K.shape[1:]), np.zeros(K.shape[1:])
    if not len(K):
        return d_q, d_k, d_v
    lse = attention(q, K, V, scale)[1]
    for h in range(q.shape[0]):
        g = h // group
        p = np.exp(scale * K[:, g] @ q[h] - lse[h])
        dp = V[:, g] @ d_ctx[h]
        ds = p * (dp - p @ dp)
        d_q[h] = scale * ds @ K[:, g]
        d_k[g] += scale * ds[-1] * q[h]
        d_v[g] += p[-1] * d_ctx[h]
    return d_q, d_k, d_v
