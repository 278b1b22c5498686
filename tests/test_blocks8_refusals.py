"""Host-side refusals of the calls on 8-bit blocks: they return before any device work."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from transformer_layer_backward_gb300 import build, _abi
    build.build()
    return _abi.load()


p, odd = C.c_void_p(256), C.c_void_p(264)


def test_quantize(lib):
    from transformer_layer_backward_gb300 import _abi as A

    def call(t=A.W_F32, x=p, rows=4, cols=8, block=1, q=p, s=p):
        return lib.tlb_fp8_quantize(t, x, rows, cols, block, q, s, None)

    for bad in (dict(t=A.W_TERNARY_I8), dict(rows=-1), dict(cols=-1), dict(block=2), dict(block=0), dict(x=None), dict(q=None),
                dict(s=None), dict(x=C.c_void_p(258)), dict(s=C.c_void_p(258)), dict(t=A.W_BF16, x=C.c_void_p(257))):
        assert call(**bad) == A.TLB_EINVAL, bad
    assert call(rows=1 << 41) == A.TLB_EUNSUPPORTED and call(rows=1 << 30, cols=1 << 30) == A.TLB_EUNSUPPORTED
    assert call(rows=0) == A.TLB_OK and call(cols=0, x=None) == A.TLB_OK


def test_linear(lib):
    from transformer_layer_backward_gb300 import _abi as A

    def call(W=p, ws=p, dY=p, ys=p, S=4, out=32, dim=48, t=A.W_F32, dX=p, w=p, n=1 << 40):
        return lib.tlb_linear_fp8_backward(W, ws, dY, ys, S, out, dim, t, dX, 0, w, n, None)

    for bad in (dict(t=2), dict(S=-1), dict(out=-1), dict(dim=-1), dict(W=None), dict(ws=None), dict(dY=None), dict(ys=None),
                dict(dX=None), dict(W=odd), dict(dY=odd), dict(dX=odd), dict(w=None), dict(n=8), dict(w=C.c_void_p(384))):
        assert call(**bad) == A.TLB_EINVAL, bad
    for name in ("S", "out", "dim"):
        assert call(**{name: (1 << 24) + 1}) == A.TLB_EUNSUPPORTED
    assert call(S=0) == A.TLB_OK and call(dim=0) == A.TLB_OK
    size = lib.tlb_linear_fp8_workspace_bytes
    assert size(-1, 1, 1) == 0 and size(1, 1 << 25, 1) == 0 and size(0, 0, 0) >= 256


def test_cache(lib):
    from transformer_layer_backward_gb300 import _abi as A

    def cache(k=256, v=256, ks=256, vs=256, n=64, kv=2, hd=64):
        return A.Kv8(k, v, ks, vs, n, kv, hd)

    def write(c, t=A.W_F32, k=p, v=p, slots=p, rows=3):
        return lib.tlb_kv8_write(C.byref(c) if c else None, t, k, 128, 64, v, 128, 64, slots, rows, None)

    def read(c, t=A.W_F32, k=p, v=p, slots=p, rows=3):
        return lib.tlb_kv8_read(C.byref(c) if c else None, slots, rows, t, k, v, 128, 64, None)

    def fwd(c, pages=p, max_pages=4, page=16, lengths=p, n=2, longest=64, heads=4, scale=0.1, t=A.W_F32, q=p, ctx=p, lse=p, w=p,
            size=1 << 40, k=None, v=None):
        return lib.tlb_kv8_attn_forward(C.byref(c) if c else None, pages, max_pages, page, lengths, n, longest, heads, scale, t, q,
                                        ctx, lse, w, size, None)

    def bwd(c, pages=p, max_pages=4, page=16, lengths=p, n=2, longest=64, heads=4, scale=0.1, t=A.W_F32, q=p, ctx=p, lse=p, w=p,
            size=1 << 40, dq=p, dk=p, dv=p):
        return lib.tlb_kv8_attn_backward(C.byref(c) if c else None, pages, max_pages, page, lengths, n, longest, heads, scale, t, q,
                                         lse, ctx, dq, dk, dv, w, size, None)

    for call in (write, read, fwd, bwd):
        assert call(None) == A.TLB_EINVAL
        for bad in (dict(k=None), dict(vs=None), dict(k=264), dict(v=264), dict(n=-1), dict(kv=0), dict(hd=0)):
            assert call(cache(**bad)) == A.TLB_EINVAL, bad
        for bad in (dict(hd=72), dict(hd=272), dict(kv=65536), dict(n=1 << 41)):
            assert call(cache(**bad)) == A.TLB_EUNSUPPORTED, bad
        assert call(cache(), t=3) == A.TLB_EINVAL
    for call in (write, read):
        for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(rows=-1)):
            assert call(cache(), **bad) == A.TLB_EINVAL, bad
        assert call(cache(), rows=1 << 40) == A.TLB_EUNSUPPORTED
        assert call(cache(), rows=0) == A.TLB_OK
    for call in (fwd, bwd):
        for bad in (dict(pages=None), dict(max_pages=-1), dict(page=0), dict(lengths=None), dict(n=-1), dict(longest=-1),
                    dict(heads=3), dict(heads=0), dict(scale=float("nan")), dict(q=None), dict(q=odd), dict(ctx=None),
                    dict(ctx=odd), dict(lse=None), dict(w=None), dict(w=C.c_void_p(384)), dict(size=100)):
            assert call(cache(), **bad) == A.TLB_EINVAL, bad
        for bad in (dict(longest=(1 << 30) + 1), dict(n=1 << 31), dict(heads=1 << 17)):
            assert call(cache(), **bad) == A.TLB_EUNSUPPORTED, bad
        assert call(cache(), n=0) == A.TLB_OK
    for name in ("dq", "dk", "dv"):
        assert bwd(cache(), **{name: None}) == A.TLB_EINVAL and bwd(cache(), **{name: odd}) == A.TLB_EINVAL
    size = lambda c, n=2, heads=4, longest=64, grad=0: lib.tlb_kv8_attn_workspace_bytes(C.byref(c), n, heads, longest, grad)
    assert size(cache(), heads=3) == 0 and size(cache(hd=72)) == 0 and size(cache(), n=-1) == 0
    assert 256 <= size(cache()) <= size(cache(), grad=1)


def test_pointers_off_their_elements(lib):
    from transformer_layer_backward_gb300 import _abi as A
    off, off4 = C.c_void_p(258), C.c_void_p(260)
    c = C.byref(A.Kv8(256, 256, 256, 256, 64, 2, 64))
    bad = C.byref(A.Kv8(256, 256, 258, 256, 64, 2, 64))
    for k, v, slots in ((off, p, p), (p, off, p), (p, p, off4)):
        assert lib.tlb_kv8_write(c, A.W_F32, k, 128, 64, v, 128, 64, slots, 3, None) == A.TLB_EINVAL
        assert lib.tlb_kv8_read(c, slots, 3, A.W_F32, k, v, 128, 64, None) == A.TLB_EINVAL
    assert lib.tlb_kv8_write(c, A.W_BF16, C.c_void_p(257), 128, 64, p, 128, 64, p, 3, None) == A.TLB_EINVAL
    assert lib.tlb_kv8_write(bad, A.W_F32, p, 128, 64, p, 128, 64, p, 3, None) == A.TLB_EINVAL
    for pages, lengths, lse in ((off, p, p), (p, off, p), (p, p, off)):
        assert lib.tlb_kv8_attn_forward(c, pages, 4, 16, lengths, 2, 64, 4, 0.1, A.W_F32, p, p, lse, p, 1 << 40, None) == A.TLB_EINVAL
        assert lib.tlb_kv8_attn_backward(c, pages, 4, 16, lengths, 2, 64, 4, 0.1, A.W_F32, p, lse, p, p, p, p, p, 1 << 40,
                                         None) == A.TLB_EINVAL
    for ws, ys in ((off, p), (p, off)):
        assert lib.tlb_linear_fp8_backward(p, ws, p, ys, 4, 32, 48, A.W_F32, p, 0, p, 1 << 40, None) == A.TLB_EINVAL


def test_binding_refuses(lib):
    """Wrong types, shapes and places are refused before the library is called."""
    import torch
    import transformer_layer_backward_gb300 as tlb
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="CUDA"):
        tlb.fp8_quantize(x)
    with pytest.raises(TypeError):
        tlb.fp8_quantize(x.double())
    with pytest.raises(ValueError):
        tlb.fp8_quantize(x[0])
    e4m3 = torch.float8_e4m3fn
    W, dY = torch.zeros(32, 256).to(e4m3), torch.zeros(4, 256).to(e4m3)
    with pytest.raises(ValueError, match="accumulate"):
        tlb.linear_fp8_backward(W, torch.ones(1, 2), dY, torch.ones(4, 2), accumulate=True, ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match=r"\[S, out\]"):
        tlb.linear_fp8_backward(W, torch.ones(1, 2), dY[:, :128], torch.ones(4, 1))
    with pytest.raises(TypeError):
        tlb.linear_fp8_backward(x, torch.ones(1, 2), dY, torch.ones(4, 2), ws=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        tlb.kv8_cache(8, 2, 64, device="cpu")


def test_struct_layout(tmp_path):
    import os
    import shutil
    import subprocess
    from transformer_layer_backward_gb300 import _abi as A
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    fields = [f[0] for f in A.Kv8._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tlb.h"\nint main(void) { printf("%zu", sizeof(tlb_kv8));'
                   + "".join('printf(" %%zu", offsetof(tlb_kv8, %s));' % f for f in fields) + "return 0; }")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(n) for n in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(A.Kv8)] + [getattr(A.Kv8, f).offset for f in fields]
