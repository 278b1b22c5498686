"""Workspace sizes of the linear-head cross entropy (host side)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from transformer_layer_backward_gb300 import build, _abi
    build.build()
    return _abi.load()


def test_the_loss_alone_needs_little(lib):
    from transformer_layer_backward_gb300 import _abi as A
    f32, bf16 = A.W_F32, A.W_BF16
    loss, both = lib.tlb_xent_forward_workspace_bytes, lib.tlb_xent_workspace_bytes
    # one token: a (max, sum) pair for 32 rows of each of four CTAs an SM, or of the head's 128-column tiles' halves
    assert 0 < loss(bf16, bf16, 1, 131072, 2560) <= 1 << 20 < both(bf16, bf16, 1, 131072, 2560, 0)
    # 2048 rows: the pairs of 2 x 1024 tiles, 8 bytes each, for every row
    assert loss(bf16, bf16, 2048, 131072, 2560) <= 8 * 2048 * 2 * 1024 * 1.01 + 65536 < both(bf16, bf16, 2048, 131072, 2560, 0) / 10
    for types in ((bf16, bf16), (f32, bf16), (f32, f32)):
        for rows, vocab, dim in ((0, 5, 8), (1, 1, 1), (7, 300, 65), (600, 5000, 33), (20000, 1000, 64)):
            assert 0 < loss(*types, rows, vocab, dim) <= both(*types, rows, vocab, dim, 0) <= both(*types, rows, vocab, dim, 1)


def test_refused_sizes_are_0(lib):
    from transformer_layer_backward_gb300 import _abi as A
    loss = lib.tlb_xent_forward_workspace_bytes
    assert loss(A.W_BF16, A.W_F32, 4, 8, 16) == 0 and loss(A.W_BF16, A.W_BF16, 4, 0, 16) == 0
    assert loss(A.W_BF16, A.W_BF16, -1, 8, 16) == 0 and loss(A.W_TERNARY_I8, A.W_BF16, 4, 8, 16) == 0
