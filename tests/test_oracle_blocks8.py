"""Pins of the oracle's 8-bit blocks and single-token attention: worked values, torch's own e4m3, and
central differences."""
import numpy as np
import pytest

from oracle import blocks8


def test_e4m3_codes_are_torchs():
    import torch
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, blocks8.E4M3, equal_nan=True)
    x = np.concatenate([np.random.default_rng(0).normal(0, s, 4000) for s in (1e-3, 0.03, 1.0, 60.0)])
    # and the borders between two codes, where the even one is taken
    x = np.concatenate([x, (blocks8.E4M3[:126] + blocks8.E4M3[1:127]) / 2]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    assert np.array_equal(blocks8.to_e4m3(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_block_scales():
    for top, want in ((448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.0, 2.0 ** -126), (1.75, 2.0 ** -8),
                      (1.76, 2.0 ** -7), (1e-45, 2.0 ** -126), (3e38, 2.0 ** 120)):
        assert blocks8.block_scale([0.0, -top, top / 2]) == want, top
    assert np.isnan(blocks8.block_scale([1.0, np.inf])) and np.isnan(blocks8.block_scale([np.nan, 1.0]))


def test_quantize_is_near_and_whole_in_blocks():
    x = np.random.default_rng(1).normal(size=(130, 200)) * np.exp(np.random.default_rng(2).normal(size=(130, 1)))
    for rows in (1, 128):
        v, s = blocks8.quantize(x, rows)
        assert s.shape == (-(-130 // rows), 2)
        full = blocks8.spread(s, rows, *x.shape)
        # half a step of 3 bits after the leading one, or of the smallest step 2^-9
        assert np.all(np.abs(v * full - x) <= np.maximum(np.abs(x) * 2.0 ** -4, full * 2.0 ** -10))


@pytest.mark.parametrize("nh,nkv,hd,n", [(1, 1, 4, 1), (4, 2, 6, 5), (6, 2, 8, 9)])
def test_attention_gradients_match_finite_differences(nh, nkv, hd, n):
    r = np.random.default_rng(3)
    q, K, V, g = (r.normal(size=s) for s in ((nh, hd), (n, nkv, hd), (n, nkv, hd), (nh, hd)))
    d_q, d_k, d_v = blocks8.attention_backward(q, K, V, g, 0.4)
    eps = 1e-6

    def check(x, dx, at):
        for i in np.ndindex(dx.shape):
            up, down = x.copy(), x.copy()
            up[at + i] += eps
            down[at + i] -= eps
            f = lambda y: float(np.sum(g * blocks8.attention(y if x is q else q, y if x is K else K, y if x is V else V, 0.4)[0]))
            # central difference: eps^2 f'''/6 ~ 1e-12 plus rounding 1e-16 |f| / eps ~ 1e-9
            assert abs((f(up) - f(down)) / (2 * eps) - dx[i]) < 1e-7

    check(q, d_q, ())
    check(K, d_k, (n - 1,))
    check(V, d_v, (n - 1,))


def test_attention_closed_forms():
    ctx, lse = blocks8.attention(np.ones((2, 4)), np.zeros((3, 1, 4)), np.arange(12.0).reshape(3, 1, 4), 1.0)
    assert np.allclose(ctx, [[4, 5, 6, 7]] * 2) and np.allclose(lse, np.log(3))
    ctx, lse = blocks8.attention(np.ones((2, 4)), np.zeros((0, 1, 4)), np.zeros((0, 1, 4)), 1.0)
    assert np.all(ctx == 0) and np.all(lse == -np.inf)
