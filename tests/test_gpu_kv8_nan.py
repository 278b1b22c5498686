"""What a value of the 8-bit cache that is NaN reaches in the attention's results and gradients, and what not."""
import pytest

from tests.test_gpu_kv8 import problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 96, 256])
@pytest.mark.parametrize("n", [1, 37, 700])
def test_a_newest_value_that_is_nan(lib, n, hd):
    """d_v = p d_ctx does not look at the values: it is what it is with a finite newest value.  ctx, d_q and d_k are NaN
    (of one key alone d_q and d_k are 0)."""
    import torch
    cache, q, g, pages, lens, longest, K, V = problem(lib, [n, 20], 10, 2, hd, 16, seed=n)
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    clean = lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g)
    j = n - 1
    slot = int(pages[0, j // 16]) * 16 + j % 16
    nan = torch.full((1, 2, hd), float("nan"), device="cuda")
    nan[:, 1] = 1.0                                            # the other KV head's stays finite
    k, _ = lib.kv8_read(cache, torch.tensor([slot], device="cuda"))
    scale = cache.tensors[1][:, slot].clone()
    lib.kv8_write(cache, k, nan, torch.tensor([slot], device="cuda"))
    cache.tensors[1][:, slot] = scale
    cache.tensors[0][slot] = torch.where(k[0] == 0, k[0], k[0] / scale[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(lib.kv8_read(cache, torch.tensor([slot], device="cuda"))[0], k)
    ctx2, lse2 = lib.kv8_attn_forward(cache, q, pages, 16, lens, longest)
    assert torch.equal(lse2, lse) and torch.all(ctx2[0, :5].isnan()) and torch.all(ctx2[0, 5:].isfinite())
    d_q, d_k, d_v = lib.kv8_attn_backward(cache, q, pages, 16, lens, longest, lse, g)
    assert torch.equal(d_v, clean[2])
    assert all(torch.equal(a[1], b[1]) for a, b in zip((ctx2, d_q, d_k), (ctx, *clean[:2])))
    if n > 1:
        assert torch.all(d_q[0, :5].isnan()) and torch.all(d_k[0, 0].isnan())
    assert torch.all(d_q[0, 5:].isfinite()) and torch.all(d_k[0, 1].isfinite())
