"""Sizes that do not fit the C ABI's 32-bit arguments are refused by the binding: ctypes would pass their low 32 bits."""
import pytest
import torch


@pytest.fixture(scope="module")
def tlb():
    import transformer_layer_backward_gb300 as tlb
    from transformer_layer_backward_gb300 import build
    build.build()
    return tlb


@pytest.mark.parametrize("block_rows", [1 << 31, (1 << 32) + 1, (1 << 32) + 128, 128 - (1 << 32)])
def test_block_rows(tlb, block_rows):
    """2^32 + 1 arrived as 1: a scale for each row, in a tensor made for one block of all rows."""
    with pytest.raises(ValueError, match="block_rows does not fit"):
        tlb.fp8_quantize(torch.zeros(4, 256), block_rows)


@pytest.mark.parametrize("page", [1 << 31, (1 << 32) + 16, 16 - (1 << 32)])
def test_page(tlb, page):
    from transformer_layer_backward_gb300 import _abi as A
    cache = A.Kv8(256, 256, 256, 256, 64, 2, 64)
    cache.device = torch.device("cpu")
    q, lse = torch.zeros(1, 4, 64), torch.zeros(1, 4)
    pages, lengths = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="page does not fit"):
        tlb.kv8_attn_forward(cache, q, pages, page, lengths, 64, ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="page does not fit"):
        tlb.kv8_attn_backward(cache, q, pages, page, lengths, 64, lse, q, ws=torch.zeros(256, dtype=torch.uint8))
