"""The linear-head cross entropy as it is called: what the binding allocates by itself."""
import pytest

from tests.test_gpu_xent import dev, problem

pytestmark = pytest.mark.gpu


@pytest.fixture
def default_dtype():
    import torch
    before = torch.get_default_dtype()
    yield torch.set_default_dtype
    torch.set_default_dtype(before)


@pytest.mark.parametrize("name", ["bfloat16", "float64"])
def test_outputs_do_not_follow_the_default_dtype(lib, default_dtype, name):
    import torch
    th, tw, _, _, t, g = problem(9, 300, 64, ("bf16", "bf16"))
    tt, tg = torch.from_numpy(t).cuda(), dev(g)
    loss, lse = lib.xent_forward(th, tw, tt)
    dh, dw = lib.xent_backward(th, tw, tt, lse, tg, grad_w=True)
    W = torch.randn(64, 32, device="cuda")
    dX = lib.linear_backward("f32", W, torch.ones(3, 32, device="cuda"))
    dY = torch.ones(3, 32, device="cuda")
    default_dtype(getattr(torch, name))
    loss2, lse2 = lib.xent_forward(th, tw, tt)
    dh2, dw2 = lib.xent_backward(th, tw, tt, lse2, tg, grad_w=True)
    dX2 = lib.linear_backward("f32", W, dY)
    for a, b in ((loss, loss2), (lse, lse2), (dh, dh2), (dw, dw2), (dX, dX2)):
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("types,rows", [(("bf16", "bf16"), 1), (("bf16", "bf16"), 300), (("f32", "bf16"), 40), (("f32", "f32"), 600)])
def test_a_workspace_for_the_loss_alone(lib, types, rows):
    import torch
    th, tw, _, _, t, g = problem(rows, 3000, 72, types)
    tt = torch.from_numpy(t).cuda()
    loss, lse = lib.xent_forward(th, tw, tt)
    ws = lib.xent_workspace(th.dtype, tw.dtype, rows, 3000, 72, grad=False)
    assert ws.numel() < lib.xent_workspace(th.dtype, tw.dtype, rows, 3000, 72).numel()
    loss2, lse2 = lib.xent_forward(th, tw, tt, ws=ws)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    lib.workspace_status(ws)
    with pytest.raises(lib.TlbError, match="workspace"):
        lib.xent_backward(th, tw, tt, lse, dev(g), ws=ws)


def test_scoring_a_token_without_a_workspace_allocates_little(lib):
    """Of its own, one token under a head of 16384 columns needs the pairs of 32 rows: less than a MB (the
    gradient's split tiles alone would be 40 MB)."""
    import torch
    th, tw, _, _, t, _ = problem(1, 16384, 64, ("bf16", "bf16"))
    tt = torch.from_numpy(t).cuda()
    lib.xent_forward(th, tw, tt)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    lib.xent_forward(th, tw, tt)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 20
