"""Host-side refusals of the linear-head cross entropy: they return before any device work."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from transformer_layer_backward_gb300 import build, _abi
    build.build()
    return _abi.load()


def test_xent_host_side_errors(lib):
    from transformer_layer_backward_gb300 import _abi as A
    p, f32, bf16 = C.c_void_p(256), A.W_F32, A.W_BF16

    def fwd(ht=bf16, h=p, wt=bf16, w=p, t=p, rows=4, vocab=8, dim=16, loss=p, lse=p, ws=p, n=1 << 40):
        return lib.tlb_xent_forward(ht, h, wt, w, t, rows, vocab, dim, loss, lse, ws, n, None)

    def bwd(ht=bf16, h=p, wt=bf16, w=p, t=p, lse=p, g=p, rows=4, vocab=8, dim=16, dh=p, dw=None, ws=p, n=1 << 40):
        return lib.tlb_xent_backward(ht, h, wt, w, t, lse, g, rows, vocab, dim, dh, dw, ws, n, None)

    for call in (fwd, bwd):
        assert call(ht=A.W_TERNARY_I8) == A.TLB_EINVAL
        assert call(wt=7) == A.TLB_EINVAL
        assert call(ht=bf16, wt=f32) == A.TLB_EUNSUPPORTED
        assert call(rows=-1) == A.TLB_EINVAL
        assert call(vocab=0) == A.TLB_EINVAL
        assert call(dim=0) == A.TLB_EINVAL
        assert call(rows=(1 << 24) + 1) == A.TLB_EUNSUPPORTED
        assert call(vocab=(1 << 24) + 1) == A.TLB_EUNSUPPORTED
        assert call(dim=(1 << 20) + 1) == A.TLB_EUNSUPPORTED
        for name in ("h", "w", "t", "lse", "ws"):
            assert call(**{name: None}) == A.TLB_EINVAL, name
        for name in ("h", "w"):
            assert call(**{name: C.c_void_p(264)}) == A.TLB_EINVAL, name
            assert b"aligned" in lib.tlb_last_error()
        assert call(ws=C.c_void_p(384)) == A.TLB_EINVAL
        assert call(n=1000) == A.TLB_EINVAL
        assert b"workspace" in lib.tlb_last_error()
        assert call(rows=0) == A.TLB_OK                     # no rows: nothing to do
    assert fwd(loss=None) == A.TLB_EINVAL
    assert bwd(g=None) == A.TLB_EINVAL and bwd(dh=None) == A.TLB_EINVAL


def test_xent_workspace_sizes(lib):
    from transformer_layer_backward_gb300 import _abi as A
    size = lambda ht, wt, rows, vocab, dim, gw=0: lib.tlb_xent_workspace_bytes(ht, wt, rows, vocab, dim, gw)
    assert size(A.W_BF16, A.W_F32, 4, 8, 16) == 0 and size(A.W_BF16, A.W_BF16, 4, 0, 16) == 0
    small, large = (size(A.W_BF16, A.W_BF16, n, 131072, 2560) for n in (1, 2048))
    assert 0 < small < large < (1 << 30)
    # dz of a whole vocabulary would not fit: pieces keep it near 512 MB
    assert size(A.W_BF16, A.W_BF16, 65536, 131072, 2560) < (5 << 29)
    # a float32 head is copied as three terms past 512 rows only
    assert size(A.W_F32, A.W_F32, 513, 1000, 64) > size(A.W_F32, A.W_BF16, 513, 1000, 64)
    assert size(A.W_F32, A.W_F32, 512, 1000, 64) == size(A.W_F32, A.W_BF16, 512, 1000, 64)
    assert size(A.W_BF16, A.W_BF16, 512, 1000, 64, 1) > size(A.W_BF16, A.W_BF16, 512, 1000, 64)
