"""Results of the linear-head cross entropy that are known without a tolerance for sums: rows
whose target is certain.

The target's logit of row i is a_i > 0 and every other one -a_i, all single products that no
type rounds.  For a_i >= 12 the true loss is log(1 + (vocab - 1) exp(-2 a_i)) <= 4e-8, and
lse = a_i + loss rounds to a_i: half a step of a float32 in [8, 16) is 4.8e-7, of a larger one
more.
"""
import numpy as np
import pytest

from tests.helpers import host
from tests.test_gpu_xent import TYPES, dev

pytestmark = pytest.mark.gpu

# rows that reach the one-pass kernel, the products on single CTAs (a float32 head: taken apart
# inside them) and on CTA pairs (a float32 head: packed)
ROWS = [1, 3, 7, 40, 100, 300, 600]
# the step of a_i and of a_i log2(e) is the same below 1.386 of a power of two, and twice as large beyond
RANGES = [(12, 16), (17, 22), (23, 32), (12000, 16000), (17000, 22000)]


def certain(rows, vocab, dim, types, low, high, column):
    rs = np.random.default_rng(rows + int(low))
    a = rs.uniform(low, high, rows).astype(np.float32)
    h, w = np.zeros((rows, dim), np.float32), np.zeros((vocab, dim), np.float32)
    h[:, dim // 2], w[:, dim // 2] = a, -1.0
    w[column, dim // 2] = 1.0
    th, tw = dev(h, types[0]), dev(w, types[1])
    return th, tw, host(th)[:, dim // 2]


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_certain_rows(lib, types, low, high):
    import torch
    vocab, dim, column = 900, 72, 517
    for rows in ROWS:
        th, tw, a = certain(rows, vocab, dim, types, low, high, column)
        tt = torch.full((rows,), column, device="cuda")
        loss, lse = lib.xent_forward(th, tw, tt)
        truth = np.log1p((vocab - 1) * np.exp(-2 * a))
        assert np.array_equal(host(lse), a), rows
        # the sum 1 + (vocab - 1) exp(-2a) and its log: a step of a float32 just above 1, 2^-23
        assert host(loss).min() >= 0.0 and np.abs(host(loss) - truth).max() <= 2.0 ** -23, rows
        g = np.random.default_rng(rows).uniform(0.2, 1.5, rows).astype(np.float32)
        dh, _ = lib.xent_backward(th, tw, tt, lse, dev(g))
        # p - 1 of the target is exp(a - lse) - 1 = 0, the others' dz g exp(-2a): sums of positive terms,
        # off by the exponential's 2^-22 and 2 a 2^-24 of its exponent, by at most 2^-8 twice in bf16
        ref = np.zeros((rows, dim))
        ref[:, dim // 2] = -g * (vocab - 1) * np.exp(-2 * a)
        off = 1e-5 if types[0] == "f32" else 2.0 ** -7
        assert np.all(np.abs(host(dh) - ref) <= off * np.abs(ref) + 1e-38), rows


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_one_column_is_certain(lib, types):
    """vocab = 1: lse is the logit itself and the loss 0, whatever the logit."""
    import torch
    for rows in ROWS:
        rs = np.random.default_rng(rows)
        th = dev(rs.normal(size=(rows, 136)).astype(np.float32) * 3, types[0])
        tw = dev(rs.normal(size=(1, 136)).astype(np.float32), types[1])
        loss, _ = lib.xent_forward(th, tw, torch.zeros(rows, dtype=torch.int64, device="cuda"))
        assert not bool(loss.any()), rows
