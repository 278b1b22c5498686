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


def test_status_of_workspaces_that_calls_make(lib, monkeypatch):
    """What a kernel records in a workspace that the caller never sees is reported by
    workspace_status() without one, once.  The record is planted from the host."""
    import torch
    th, tw, _, _, t, g = problem(12, 300, 64, ("bf16", "bf16"))
    tt, tg = torch.from_numpy(t).cuda(), dev(g)
    lib.workspace_status()
    make = lib.api.xent_workspace
    for plant in ([0], [1], [0, 1]):                             # which of the two calls' records
        left = []

        def planted(*args, **kw):
            ws = make(*args, **kw)
            if len(left) in plant:
                ws[:8].view(torch.int32).copy_(torch.tensor([1, 77], dtype=torch.int32))   # a wait, its site
            left.append(ws)
            return ws

        monkeypatch.setattr(lib.api, "xent_workspace", planted)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        loss, lse = lib.xent_forward(th, tw, tt, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        lib.xent_backward(th, tw, tt, lse, tg)
        monkeypatch.setattr(lib.api, "xent_workspace", make)
        lib.xent_forward(th, tw, tt)                             # a later call in order does not hide it
        with pytest.raises(lib.TlbError, match="wait ran out.*77") as e:
            lib.workspace_status()
        assert e.value.code == lib._abi.TLB_ETIMEOUT
        lib.workspace_status()


def test_only_the_status_block_is_cleared(lib):
    """A workspace holding anything but for its status block gives the same bits."""
    import torch
    for types, rows in ((("bf16", "bf16"), 2), (("bf16", "bf16"), 50), (("bf16", "bf16"), 300), (("f32", "bf16"), 300),
                        (("f32", "f32"), 7), (("f32", "f32"), 300), (("f32", "f32"), 600)):
        th, tw, _, _, t, g = problem(rows, 1500, 72, types)
        tt, tg = torch.from_numpy(t).cuda(), dev(g)
        got = []
        for fill in (0, 255):                                    # zeros; NaN wherever a float is read
            ws = lib.xent_workspace(th.dtype, tw.dtype, rows, 1500, 72, grad_w=True)
            ws[256:] = fill
            loss, lse = lib.xent_forward(th, tw, tt, ws=ws)
            ws[256:] = fill
            dh, dw = lib.xent_backward(th, tw, tt, lse, tg, grad_w=True, ws=ws)
            got.append((loss, lse, dh, dw))
            lib.workspace_status(ws)
        assert all(torch.equal(a, b) for a, b in zip(*got)), (types, rows)


def test_calls_without_a_workspace_in_a_captured_graph(lib):
    import torch
    th, tw, _, _, t, g = problem(40, 900, 64, ("bf16", "bf16"))
    tt, tg = torch.from_numpy(t).cuda(), dev(g)
    loss, lse = lib.xent_forward(th, tw, tt)
    dh, _ = lib.xent_backward(th, tw, tt, lse, tg)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        loss2, lse2 = lib.xent_forward(th, tw, tt)
        dh2, _ = lib.xent_backward(th, tw, tt, lse2, tg)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dh, dh2)
    lib.workspace_status()
