"""8-bit tensors of more than 2^32 bytes: what lies behind that is found, and equal to the same rows by themselves."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    import torch
    yield
    torch.cuda.empty_cache()


def test_quantize_behind_4_gb(lib):
    import torch
    rows, cols = 70000, 65536                                  # 4.6e9 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-130:] = torch.randn(130, cols, device="cuda")
    for block_rows, last in ((1, 130), (128, rows % 128)):
        q, s = lib.fp8_quantize(x, block_rows)
        want, want_s = lib.fp8_quantize(x[-last:].contiguous(), block_rows)
        assert torch.equal(q[-last:].view(torch.uint8), want.view(torch.uint8))
        assert torch.equal(s[-want_s.shape[0]:], want_s)
        assert torch.count_nonzero(q[:1000].view(torch.uint8)) == 0
        del q, s


@pytest.mark.parametrize("S", [3, 40])
def test_linear_with_a_weight_behind_4_gb(lib, S):
    import torch
    out, dim, last = 8192, 600064, 512                         # 4.9e9 weights
    W = torch.zeros(dim, out, dtype=torch.uint8, device="cuda")
    W[-last:] = torch.randint(0, 0x7F, (last, out), dtype=torch.uint8, device="cuda")
    W = W.view(torch.float8_e4m3fn)
    w_s = torch.rand(dim // 128, out // 128, device="cuda") + 0.5
    dY, y_s = lib.fp8_quantize(torch.randn(S, out, device="cuda"))
    got = lib.linear_fp8_backward(W, w_s, dY, y_s)
    want = lib.linear_fp8_backward(W[-last:].contiguous(), w_s[-(last // 128):].contiguous(), dY, y_s)
    # the same terms; how the columns are shared out, and with it the order of the last few sums, goes by the sizes
    assert (got[:, -last:] - want).norm() <= 1e-6 * want.norm()
    assert torch.count_nonzero(got[:, :-last]) == 0
    lib.workspace_status()


def test_cache_behind_4_gb(lib):
    import torch
    n, kv, hd, keys = 2200000, 8, 256, 300                     # 4.5e9 bytes of keys, and of values
    cache, small = lib.kv8_cache(n, kv, hd), lib.kv8_cache(keys, kv, hd)
    k, v = torch.randn(keys, kv, hd, device="cuda"), torch.randn(keys, kv, hd, device="cuda")
    slots, own = torch.arange(n - keys, n, device="cuda"), torch.arange(keys, device="cuda")
    lib.kv8_write(cache, k, v, slots)
    lib.kv8_write(small, k, v, own)
    assert all(torch.equal(a, b) for a, b in zip(lib.kv8_read(cache, slots), lib.kv8_read(small, own)))
    q, g = torch.randn(1, 8, hd, device="cuda"), torch.randn(1, 8, hd, device="cuda")
    lens = torch.tensor([keys], dtype=torch.int32, device="cuda")
    far = (slots // 4).unique().to(torch.int32)[None]          # n - keys is a multiple of the page of 4
    near = torch.arange(keys // 4, dtype=torch.int32, device="cuda")[None]
    a = lib.kv8_attn_forward(cache, q, far, 4, lens, keys)
    b = lib.kv8_attn_forward(small, q, near, 4, lens, keys)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = lib.kv8_attn_backward(cache, q, far, 4, lens, keys, a[1], g)
    b = lib.kv8_attn_backward(small, q, near, 4, lens, keys, b[1], g)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
