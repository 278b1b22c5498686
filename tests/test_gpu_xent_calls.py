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
