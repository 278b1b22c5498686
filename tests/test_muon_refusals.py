"""Host-side refusals of the Muon step: they return before any device work."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from transformer_layer_backward_gb300 import build, _abi
    build.build()
    return _abi.load()


def test_muon_host_side_errors(lib):
    from transformer_layer_backward_gb300 import _abi as A
    p = 256

    def call(mats, steps=5, eps=1e-7, ws=C.c_void_p(256), n_bytes=1 << 40, n=None, cfg=True):
        arr = (A.MuonMat * max(len(mats), 1))(*mats)
        c = A.MuonCfg(0.1, 0.95, 0.0, eps, 3.4445, -4.775, 2.0315, steps, 1)
        return lib.tlb_muon(arr, len(mats) if n is None else n, C.byref(c) if cfg else None, ws, n_bytes, None)

    ok = A.MuonMat(p, p, p, 4, 8, 1.0, 1.0)
    assert call([ok], cfg=False) == A.TLB_EINVAL
    assert call([ok], steps=0) == A.TLB_EINVAL and call([ok], steps=101) == A.TLB_EINVAL
    assert call([ok], eps=-1.0) == A.TLB_EINVAL and call([ok], eps=float("nan")) == A.TLB_EINVAL
    assert call([ok], n=-1) == A.TLB_EINVAL
    assert call([A.MuonMat(p, p, p, -1, 8, 1.0, 1.0)]) == A.TLB_EINVAL
    assert call([ok, A.MuonMat(p, p, p, 65, 65, 1.0, 1.0)]) == A.TLB_EUNSUPPORTED
    assert b"matrix 1" in lib.tlb_last_error()
    assert call([A.MuonMat(p, p, p, (1 << 24) + 1, 4, 1.0, 1.0)]) == A.TLB_EUNSUPPORTED
    for i in range(3):
        ptr = [p, p, p]
        ptr[i] = None
        assert call([A.MuonMat(*ptr, 4, 8, 1.0, 1.0)]) == A.TLB_EINVAL
    assert call([ok], ws=None) == A.TLB_EINVAL
    assert call([ok], ws=C.c_void_p(264)) == A.TLB_EINVAL
    assert call([ok], n_bytes=300) == A.TLB_EINVAL
    assert b"workspace" in lib.tlb_last_error()
    assert call([]) == A.TLB_OK                                        # nothing to do
    assert call([A.MuonMat(None, None, None, 0, 8, 1.0, 1.0)], ws=None, n_bytes=0) == A.TLB_OK


def test_muon_workspace_and_structs(lib, tmp_path):
    from transformer_layer_backward_gb300 import _abi as A
    size = lambda *shapes: lib.tlb_muon_workspace_bytes(
        (A.MuonMat * len(shapes))(*[A.MuonMat(None, None, None, r, c, 1.0, 1.0) for r, c in shapes]), len(shapes))
    assert size((65, 65)) == 0 and 0 < size((4, 8)) < size((4, 8), (16, 2560)) < size((64, 2560))
    assert size((2560, 16)) == size((16, 2560))
    import shutil
    import subprocess
    import os
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tlb.h"\nint main(void) {\n'
                   'printf("%zu %zu %zu %zu %zu\\n", sizeof(tlb_muon_mat), offsetof(tlb_muon_mat, cols),'
                   ' offsetof(tlb_muon_mat, scale), sizeof(tlb_muon_cfg), offsetof(tlb_muon_cfg, nesterov));\nreturn 0; }\n')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(A.MuonMat), A.MuonMat.cols.offset, A.MuonMat.scale.offset, C.sizeof(A.MuonCfg),
                   A.MuonCfg.nesterov.offset]
