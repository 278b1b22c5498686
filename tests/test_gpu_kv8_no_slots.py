"""Attention over a cache that holds no slot: every row is empty, whatever lengths and pages say."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 256])
def test_no_slots(lib, hd):
    import torch
    cache = lib.kv8_cache(0, 2, hd)
    q = torch.randn(3, 4, hd, device="cuda")
    pages = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 0, 32], dtype=torch.int32, device="cuda")
    ctx, lse = lib.kv8_attn_forward(cache, q, pages, 16, lens, 32)
    assert torch.all(ctx == 0) and torch.all(lse == -float("inf"))
    for grad in lib.kv8_attn_backward(cache, q, pages, 16, lens, 32, lse, torch.randn_like(q)):
        assert torch.all(grad == 0)
    slots = torch.tensor([0, 5], device="cuda")
    lib.kv8_write(cache, q[:2, :2], q[:2, 2:], slots)          # every slot is outside: nothing to write
    assert all(torch.count_nonzero(x) == 0 for x in lib.kv8_read(cache, slots))
