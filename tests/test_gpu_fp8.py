"""8-bit blocks on the GPU: quantised bit for bit as the float64 oracle does it, and the transposed-weight
product of operands held that way.

Tolerance of the product: the products of e4m3 values are exact, a sum of n terms in float32 is off by at
most n 2^-24 of the sum of their magnitudes where each addition is rounded to nearest, and by twice that where
bits are cut off; n = 128 within a block, one a block after that, and three roundings of the scales, of a
float32 or bf16 result (half a step, 2^-24 or 2^-8 of it) on top.
"""
import numpy as np
import pytest

from oracle import blocks8
from tests.helpers import check, host

pytestmark = pytest.mark.gpu


def floats(rows, cols, seed=0, spread=2.0):
    r = np.random.default_rng(seed)
    return (r.normal(size=(rows, cols)) * np.exp(r.normal(0, spread, (rows, 1)) - 3)).astype(np.float32)


def dev(x, bf16=False):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.bfloat16() if bf16 else t


def same(q, scales, x, block_rows):
    values, want = blocks8.quantize(host(x), block_rows)
    assert np.array_equal(host(scales), want, equal_nan=True)
    assert np.array_equal(host(q.float()), values, equal_nan=True)


SIZES = [(1, 1), (1, 2560), (3, 127), (5, 129), (2, 4), (130, 260), (128, 128), (257, 384), (33, 1001), (64, 72)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(lib, rows, cols, block_rows, bf16):
    x = dev(floats(rows, cols, seed=rows + cols), bf16)
    q, s = lib.fp8_quantize(x, block_rows)
    same(q, s, x, block_rows)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(lib, block_rows, bf16):
    """Blocks of zeros, of the smallest and largest floats, at the border of two scales, with infinities and NaN."""
    x = floats(140, 700, 5)
    x[:128, :128] = 0
    x[3, 130:140] = np.float32(1e-45)
    x[3, 140:256] = 0
    x[4, 128:256] *= np.float32(1e-38)
    x[5, 128:256] = np.linspace(-3e38, 3e38, 128, dtype=np.float32)
    for i, top in enumerate((448.0, 449.0, 447.0, 1.75, 1.7578125, 224.0, 0.875)):
        x[8 + i, 256:384] = np.linspace(-top, top, 128, dtype=np.float32)
    x[129, 390], x[130, 520], x[131, 699] = np.inf, -np.inf, np.nan
    x[139, 3] = np.float32(-0.0)
    t = dev(x, bf16)
    q, s = lib.fp8_quantize(t, block_rows)
    same(q, s, t, block_rows)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_tensors_that_start_anywhere(lib, block_rows, bf16):
    """A tensor, codes and scales that begin an element past an aligned place; the neighbours are left alone."""
    import torch
    rows, cols = 37, 260
    x = dev(floats(1, rows * cols + 1, 3), bf16)[0, 1:].reshape(rows, cols)
    q = torch.full((rows * cols + 2,), 7, dtype=torch.uint8, device="cuda")
    blocks = (-(-rows // block_rows), 3)
    s = torch.full((blocks[0] * 3 + 2,), 5.0, device="cuda")
    lib.fp8_quantize(x, block_rows, q=q[1:-1].view(torch.float8_e4m3fn).reshape(rows, cols), scales=s[1:-1].reshape(blocks))
    same(q[1:-1].view(torch.float8_e4m3fn).reshape(rows, cols), s[1:-1].reshape(blocks), x, block_rows)
    assert q[0] == 7 and q[-1] == 7 and s[0] == 5 and s[-1] == 5


def operands(S, out, dim, seed=0, scales="any"):
    """dY and W in blocks, their scales any floats, as device tensors."""
    import torch
    r = np.random.default_rng(seed)
    nb = -(-out // 128)
    code = lambda *shape: torch.from_numpy(r.integers(0, 255, shape, dtype=np.uint8).astype(np.uint8)).cuda()
    dY, W = code(S, out), code(dim, out)
    for t in (dY, W):
        t[(t & 0x7F) == 0x7F] = 0x38                           # the NaN codes
    ys = np.exp(r.normal(0, 1, (S, nb)) - 9).astype(np.float32)
    ws = np.exp(r.normal(0, 1, (-(-dim // 128), nb)) - 9).astype(np.float32)
    return W.view(torch.float8_e4m3fn), dev(ws), dY.view(torch.float8_e4m3fn), dev(ys)


def bound(W, ws, dY, ys, got_dtype, ref, base=None):
    import torch
    full = np.abs(host(W.float())) * blocks8.spread(host(ws), 128, *W.shape)
    mag = (np.abs(host(dY.float())) * blocks8.spread(host(ys), 1, *dY.shape)) @ full.T
    n = 128 + ws.shape[1] + 3
    half = 2.0 ** (-24 if got_dtype == torch.float32 else -8)
    return mag * n * 2.0 ** -23 + (np.abs(ref) + (0 if base is None else 2.0 ** -20 * np.abs(base))) * half * (1 + 2.0 ** -8) + 1e-45


def run_linear(lib, S, out, dim, bf16=False, add=False, seed=0, ws=None):
    import torch
    W, w_s, dY, y_s = operands(S, out, dim, seed)
    dtype = torch.bfloat16 if bf16 else torch.float32
    ref = blocks8.linear_backward(host(W.float()), host(w_s), host(dY.float()), host(y_s))
    size = max(float(np.sqrt(np.mean(ref ** 2))), 1e-30)
    base = dev(floats(S, dim, seed + 1, 0.1) * np.float32(20 * size), bf16) if add else None
    if ws is None:
        ws = lib.linear_fp8_workspace(S, out, dim)
    got = lib.linear_fp8_backward(W, w_s, dY, y_s, out=None if base is None else base.clone(), accumulate=add, dtype=dtype, ws=ws)
    lib.workspace_status(ws)
    if add:
        ref = ref + host(base)
    assert got.dtype == dtype and got.shape == (S, dim)
    err = np.abs(host(got) - ref)
    lim = bound(W, w_s, dY, y_s, dtype, ref, host(base) if add else None)
    assert np.all(np.isfinite(host(got)))
    assert np.all(err <= lim), (np.max(err / lim), np.unravel_index(np.argmax(err / lim), err.shape))
    check("dX", host(got), ref, rel_l2=1e-5 if not bf16 else 2.0 ** -8, max_abs=None)
    return got


LINEAR = [(1, 128, 128), (1, 1, 1), (1, 9728, 2560), (2, 2560, 300), (3, 130, 77), (4, 1000, 129), (7, 17, 257), (8, 4096, 512),
          (9, 384, 640), (16, 2560, 1024), (17, 1001, 333), (32, 512, 96), (33, 640, 1280), (64, 2560, 2560), (100, 1040, 1000),
          (128, 256, 128), (129, 272, 384), (200, 3000, 515), (256, 1024, 1024), (300, 48, 2304), (333, 1001, 4099),
          (512, 2048, 768), (777, 16, 16), (1030, 656, 1300)]


@pytest.mark.parametrize("S,out,dim", LINEAR)
def test_linear(lib, S, out, dim):
    run_linear(lib, S, out, dim, seed=S)


@pytest.mark.parametrize("bf16,add", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("S,out,dim", [(1, 640, 300), (5, 1001, 77), (40, 1040, 515), (130, 384, 1000), (260, 2560, 520)])
def test_linear_types_and_sums(lib, S, out, dim, bf16, add):
    run_linear(lib, S, out, dim, bf16, add, seed=S)


@pytest.mark.parametrize("S,out,dim", [(2048, 9728, 2560), (2048, 2560, 9728), (1500, 4096, 2560)])
def test_linear_large_rows_by_sample(lib, S, out, dim):
    """Full sizes, every 37th row and every 41st column against the oracle; the same bits on a second call."""
    import torch
    W, w_s, dY, y_s = operands(S, out, dim, 1)
    ws = lib.linear_fp8_workspace(S, out, dim)
    got = lib.linear_fp8_backward(W, w_s, dY, y_s, ws=ws)
    again = lib.linear_fp8_backward(W, w_s, dY, y_s, ws=ws)
    lib.workspace_status(ws)
    assert torch.equal(got, again)
    r, c = np.arange(0, S, 37), np.arange(0, dim, 41)
    full_w = host(W.float()[c]) * np.repeat(host(w_s), 128, 1)[c // 128][:, :out]
    full_y = host(dY.float()[r]) * np.repeat(host(y_s)[r], 128, 1)[:, :out]
    ref, mag = full_y @ full_w.T, np.abs(full_y) @ np.abs(full_w).T
    err = np.abs(host(got)[np.ix_(r, c)] - ref)
    assert np.all(err <= mag * (131 + -(-out // 128)) * 2.0 ** -23)
    check("dX", host(got)[np.ix_(r, c)], ref, rel_l2=1e-5, max_abs=None)


@pytest.mark.parametrize("S", [1, 6, 40, 300])
def test_linear_empty_sum(lib, S):
    import torch
    W, dY = (torch.empty(n, 0, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for n in (20, S))
    base = torch.randn(S, 20, device="cuda")
    none = torch.empty(1, 0, device="cuda")
    assert torch.equal(lib.linear_fp8_backward(W, none, dY, torch.empty(S, 0, device="cuda")), torch.zeros(S, 20, device="cuda"))
    got = lib.linear_fp8_backward(W, none, dY, torch.empty(S, 0, device="cuda"), out=base.clone(), accumulate=True)
    assert torch.equal(got, base)


@pytest.mark.parametrize("S", [3, 200])
def test_linear_nan_stays_in_its_rows_and_columns(lib, S):
    """A block of dY that is NaN makes its row NaN, one of W its 128 outputs, and nothing else."""
    import torch
    W, w_s, dY, y_s = operands(S, 640, 400, 2)
    clean = lib.linear_fp8_backward(W, w_s, dY, y_s)
    y_s[2, 1] = float("nan")
    w_s[1, 3] = float("nan")
    got = lib.linear_fp8_backward(W, w_s, dY, y_s)
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[2] = True
    bad[:, 128:256] = True
    assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("S", [1, 24, 300])
def test_linear_only_the_status_block_is_cleared(lib, S):
    import torch
    W, w_s, dY, y_s = operands(S, 1000, 700, 4)
    got = []
    for fill in (0, 255):
        ws = lib.linear_fp8_workspace(S, 1000, 700)
        ws[256:] = fill
        got.append(lib.linear_fp8_backward(W, w_s, dY, y_s, ws=ws))
        lib.workspace_status(ws)
    assert torch.equal(*got)
    assert torch.equal(got[0], lib.linear_fp8_backward(W, w_s, dY, y_s))
    lib.workspace_status()


def test_quantized_linear_against_the_bf16_product(lib):
    """As it is used: a bf16 weight quantised once, gradients as they come, against the product in floats.  Each
    e4m3 rounding is within 2^-4 of its value, so two of them within 1/8 of the sum of magnitudes, and far
    nearer in the norm (independent roundings of 2^-4 / sqrt(3) at most: 0.05 of the result's norm)."""
    S, out, dim = 96, 1024, 512
    w, g = dev(floats(dim, out, 1, 0.1), True), dev(floats(S, out, 2))
    W, w_s = lib.fp8_quantize(w, 128)
    dY, y_s = lib.fp8_quantize(g)
    got = lib.linear_fp8_backward(W, w_s, dY, y_s)
    ref = host(g) @ host(w).T
    check("dX", host(got), ref, rel_l2=0.051, max_abs=None)
