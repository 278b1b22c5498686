"""GPU parity of the linear-head cross entropy and its gradient against the float64 oracle.

Tolerances, from the arithmetic:
  * float32 results (loss and lse always; gradients of float32 hidden rows): operands exact
    (three bf16 terms), so what remains is the fp32 sums.  The tensor core cuts after every
    MMA, 80 MMAs a chunk: at most 80 x 2^-23 = 9.5e-6 of the chunk's largest partial sum, a
    tenth of that in practice.  The stated float32 bar (relative L2 1e-5, scaled max 1e-4).
  * gradients of bf16 hidden rows: dz and the result are each rounded to bf16 once, at most
    half a step, 2^-8: |error| <= 2^-8 (|dz| |w| + |result|) in every element, plus the float32
    bar.  With independent roundings of rms <= 2^-8 / sqrt(3) the two together stay under
    sqrt(2/3) 2^-8 = 3.2e-3 in relative L2 (operands without structure, so that a sum is as
    large as the root of its terms' squares): the stated bf16 bar of 5e-3.
"""
import numpy as np
import pytest

from oracle import ops
from synth import rng
from tests.helpers import BF16_REL_L2, check, errors, host

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")]
HALF = 2.0 ** -8
SHAPES = [(1, 1, 1), (1, 2, 8), (1, 7, 64), (1, 5000, 2560), (2, 300, 72), (31, 129, 63), (64, 257, 136),
          (127, 1000, 100), (128, 512, 128), (129, 511, 130), (257, 1023, 65), (300, 5003, 1001), (520, 20000, 320), (512, 700, 260), (513, 700, 260), (200, 3001, 3073),
          (130, 40, 1030), (100, 70000, 36), (20, 5, 1), (40, 1, 3)]


def normal(name, shape, std=1.0):
    n = int(np.prod(shape))
    return rng.normal(rng.stream_key(0, "xent", name, *shape), n, 0.0, std).reshape(shape).astype(np.float32)


def dev(a, kind="f32"):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16) if kind == "bf16" else t


def problem(rows, vocab, dim, types, std=0.3, seed=0):
    """Hidden rows and a head in their types (float64 copies of the rounded values), targets
    with some rows without one, per-row loss weights."""
    h, w = normal("h%d" % seed, (rows, dim)), normal("w%d" % seed, (vocab, dim), std / np.sqrt(max(dim / 64, 1)))
    th, tw = dev(h, types[0]), dev(w, types[1])
    rs = np.random.default_rng(rows * 1000003 + vocab + seed)
    t = rs.integers(0, vocab, rows)
    t[rs.uniform(size=rows) < 0.2] = -1
    if rows > 2:
        t[0], t[1], t[rows - 1] = 0, vocab - 1, vocab          # first, last, one past the last
    g = rs.uniform(0.2, 1.5, rows).astype(np.float32)
    return th, tw, host(th), host(tw), t, g


def check_gradient(name, got, ref, terms, is_bf16, dim_ok=True):
    """terms: the sum of the absolute products behind each element."""
    if not is_bf16:
        check(name, got, ref)
        return
    limit = HALF * (terms * 1.01 + np.abs(ref) * 1.01) + 1e-5 * terms + 1e-30
    assert np.all(np.isfinite(got)), name
    over = np.abs(got - ref) - limit
    assert np.all(over <= 0), "%s: %.3e over its bound" % (name, over.max())
    if ref.size >= 4096:
        rel, _ = errors(got, ref)
        assert rel <= BF16_REL_L2, "%s: relative L2 %.3e" % (name, rel)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("rows,vocab,dim", SHAPES)
def test_xent(lib, rows, vocab, dim, types):
    import torch
    th, tw, h, w, t, g = problem(rows, vocab, dim, types)
    tt = torch.from_numpy(t).cuda()
    ws = lib.xent_workspace(th.dtype, tw.dtype, rows, vocab, dim, grad_w=True)
    loss, lse = lib.xent_forward(th, tw, tt, ws=ws)
    rloss, rlse = ops.xent_forward(h, w, t)
    check("loss", host(loss), rloss)
    check("lse", host(lse), rlse)
    assert np.all(host(loss)[(t < 0) | (t >= vocab)] == 0)
    tl = dev(rlse.astype(np.float32))
    dh, dw = lib.xent_backward(th, tw, tt, tl, dev(g), grad_w=True, ws=ws)
    assert dh.dtype == th.dtype and dw.dtype == th.dtype
    lib.workspace_status(ws)
    dz = ops.xent_dlogits(h, w, t, host(tl), g)
    rdh, rdw = ops.xent_backward(h, w, t, host(tl), g)
    bf = types[0] == "bf16"
    if vocab == 1 and not bf:
        # p = 1: dz = g (exp(z - lse) - 1) is nothing but rounding.  z, a sum of dim products in fp32,
        # is (dim + 2) 2^-24 |h| |w| off at most, and dz g times that.
        off = np.where((t == 0)[:, None], g[:, None] * (dim + 2) * 2.0 ** -24 * (np.abs(h) @ np.abs(w).T), 0.0)
        assert np.all(np.abs(host(dh) - rdh) <= off @ np.abs(w))
        assert np.all(np.abs(host(dw) - rdw) <= off.T @ np.abs(h))
        return
    check_gradient("d_hidden", host(dh), rdh, np.abs(dz) @ np.abs(w), bf)
    check_gradient("d_w", host(dw), rdw, np.abs(dz).T @ np.abs(h), bf)
    only, none = lib.xent_backward(th, tw, tt, tl, dev(g), ws=ws)       # without the head's gradient
    assert none is None
    check_gradient("d_hidden alone", host(only), rdh, np.abs(dz) @ np.abs(w), bf)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("rows,vocab,dim", [(1, 1, 2), (1, 9, 6000), (1, 30011, 1026), (2, 8, 64), (2, 1237, 2560),
                                            (3, 1000, 320), (3, 5, 2), (4, 4099, 2560), (4, 12, 1022), (4, 300, 3074),
                                            (5, 2000, 2560), (1, 50, 1001), (1, 700, 2085), (2, 1003, 333), (4, 77, 5),
                                            (3, 2001, 1999), (4, 900, 511), (6, 1500, 513), (9, 500, 1216), (16, 3001, 130),
                                            (15, 600, 1025), (17, 400, 130), (12, 999, 3073), (12, 700, 832),
                                            (13, 700, 832), (10, 20011, 832), (8, 900, 1000), (7, 333, 77)])
def test_few_rows(lib, rows, vocab, dim, types):
    """Up to four rows take the one-pass kernel, and with a float32 head up to eight, in turns;
    blocks of head rows that are not full, lengths past what the registers hold, and one row
    more beside them."""
    n0 = lib.launch_count()
    test_xent(lib, rows, vocab, dim, types)
    names = lib.launch_names(n0)
    turns = [min(4, rows - r) for r in range(0, rows, 4)]
    for name, four in (("xent_token_loss", 5), ("xent_token_grad", 3)):
        fits = all(dim <= 1024 * {1: 6, 2: 5}.get(n, four) for n in turns)
        assert (name in names) == (fits and rows <= (8 if types[1] == "f32" else 4)), names
    assert ("xent_dw" in names) == ("xent_token_grad" not in names)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("rows,dim", [(1, 512), (3, 511), (40, 512), (200, 264)])
def test_confident_rows(lib, rows, dim, types):
    """Targets of probability 1 - 1e-3 and nearer: p - 1 and the loss are small differences of
    large numbers.  lse carries half a step of its own, 2^-24 x 16 = 1e-6, so 1 - p of 1e-3 is
    known to 1e-3 at best: the gradient is compared for the lse that it is given, where expm1
    leaves the target's logit: sums of 512 products in fp32, at most 2^-22 of |h| |w| = 20 in
    the terms' absolute sum, 5e-6 of p, 5e-3 of 1 - p = 1e-3."""
    import torch
    vocab = 900
    th, tw, h, w, t, g = problem(rows, vocab, dim, types)
    t[:] = np.arange(rows) % vocab
    h = h * 0.1
    h += w[t] / np.sum(w[t] ** 2, 1, keepdims=True) * 15.0     # the target's logit near 15, the others' near 0
    th = dev(h.astype(np.float32), types[0])
    h, tt = host(th), torch.from_numpy(t).cuda()
    rlse = ops.xent_forward(h, w, t)[1].astype(np.float32)
    loss, lse = lib.xent_forward(th, tw, tt)
    # half a step of lse and of the logit, 2^-24 x 16 each, and the sum's 5e-6
    assert np.max(np.abs(host(loss) - ops.xent_forward(h, w, t)[0])) <= 1e-5
    dh, _ = lib.xent_backward(th, tw, tt, dev(rlse), dev(g))
    rdh, _ = ops.xent_backward(h, w, t, host(dev(rlse)), g)
    rel, _ = errors(host(dh), rdh)
    assert rel <= (5e-3 if types[0] == "f32" else 1e-2), rel


@pytest.mark.parametrize("types,rows,vocab,dim", [(("f32", "bf16"), 2048, 50001, 64),     # pieces of dz
                                                  (("f32", "f32"), 3, 36000, 2560),      # pieces of the packed head
                                                  (("bf16", "bf16"), 6000, 50001, 40),
                                                  (("bf16", "bf16"), 20000, 600, 72)])   # row chunks of the loss
def test_pieces(lib, types, rows, vocab, dim):
    import torch
    th, tw, h, w, t, g = problem(rows, vocab, dim, types)
    tt = torch.from_numpy(t).cuda()
    loss, lse = lib.xent_forward(th, tw, tt)
    rloss, rlse = ops.xent_forward(h, w, t)
    check("loss", host(loss), rloss)
    check("lse", host(lse), rlse)
    tl = dev(rlse.astype(np.float32))
    dh, dw = lib.xent_backward(th, tw, tt, tl, dev(g), grad_w=True)
    dz = ops.xent_dlogits(h, w, t, host(tl), g)
    rdh, rdw = ops.xent_backward(h, w, t, host(tl), g)
    check_gradient("d_hidden", host(dh), rdh, np.abs(dz) @ np.abs(w), types[0] == "bf16")
    check_gradient("d_w", host(dw), rdw, np.abs(dz).T @ np.abs(h), types[0] == "bf16")


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("rows", [5, 140])
def test_rows_without_target_hold_anything(lib, types, rows):
    """NaN and infinities in the hidden rows and statistics of rows without a target reach
    nothing but those rows' lse."""
    import torch
    vocab, dim = 700, 96
    th, tw, h, w, t, g = problem(rows, vocab, dim, types)
    t[2::3] = -100
    out = t < 0
    out |= t >= vocab
    tt = torch.from_numpy(t).cuda()
    loss0, lse0 = lib.xent_forward(th, tw, tt)
    dh0, dw0 = lib.xent_backward(th, tw, tt, lse0, dev(g), grad_w=True)
    bad, keep = torch.from_numpy(out).cuda(), torch.from_numpy(~out).cuda()
    th2, lse2, g2 = th.clone(), lse0.clone(), dev(g).clone()
    th2[bad] = float("nan")
    th2[bad.nonzero()[0, 0]] = float("inf")
    loss2, lse_n = lib.xent_forward(th2, tw, tt)
    assert torch.equal(loss2, loss0) and torch.equal(lse_n[keep], lse0[keep])
    lse2[bad] = float("nan")
    g2[bad] = float("inf")
    dh2, dw2 = lib.xent_backward(th2, tw, tt, lse2, g2, grad_w=True)
    assert torch.equal(dh2, dh0) and torch.equal(dw2, dw0)
    assert bool((dh2[bad] == 0).all())
    none = torch.full_like(tt, -1)
    loss3, _ = lib.xent_forward(th, tw, none)
    dh3, dw3 = lib.xent_backward(th, tw, none, lse0, dev(g), grad_w=True)
    assert not bool(loss3.any()) and not bool(dh3.any()) and not bool(dw3.any())


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_large_logits(lib, types):
    """Logits of +-10^4: no overflow, a certain row has loss 0 and a gradient of 0."""
    import torch
    rows, vocab, dim = 6, 900, 64
    h = np.zeros((rows, dim), np.float32)
    w = np.zeros((vocab, dim), np.float32)
    h[:, 0] = [100, -100, 100, -100, 0, 1]
    w[:, 0] = np.linspace(-96, 96, vocab).astype(np.float32)
    th, tw = dev(h, types[0]), dev(w, types[1])
    t = np.array([vocab - 1, 0, 0, vocab - 1, 5, 6])
    loss, lse = lib.xent_forward(th, tw, torch.from_numpy(t).cuda())
    rloss, rlse = ops.xent_forward(host(th), host(tw), t)
    # logits up to 9600 in fp32: 2^-24 of them per rounding, a handful of roundings
    assert np.max(np.abs(host(lse) - rlse)) <= 9600 * 2.0 ** -21
    assert np.max(np.abs(host(loss) - rloss)) <= 9600 * 2.0 ** -20
    dh, _ = lib.xent_backward(th, tw, torch.from_numpy(t).cuda(), lse, dev(np.ones(rows, np.float32)))
    assert bool(torch.isfinite(dh).all())


def test_far_rows_of_a_large_head(lib):
    """Element offsets past 2^31 in W: the last vocabulary rows are read and written where they are."""
    import torch
    rows, vocab, dim = 2, 1000001, 2200
    gen = torch.Generator(device="cuda").manual_seed(1)
    tw = (torch.randn(vocab, dim, generator=gen, device="cuda", dtype=torch.bfloat16) * 0.05)
    th = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
    tt = torch.tensor([vocab - 1, 999997], device="cuda")
    g = torch.ones(rows, device="cuda")
    loss, lse = lib.xent_forward(th, tw, tt)
    z = torch.cat([th.double() @ tw[i:i + 100000].double().T for i in range(0, vocab, 100000)], 1)
    rlse = torch.logsumexp(z, 1)
    check("lse", host(lse), host(rlse))
    check("loss", host(loss), host(rlse - z.gather(1, tt[:, None])[:, 0]))
    dh, dw = lib.xent_backward(th, tw, tt, lse, g, grad_w=True)
    dz = torch.exp(z - lse.double()[:, None])
    dz[torch.arange(rows), tt] -= 1
    ref = sum(dz[:, i:i + 100000] @ tw[i:i + 100000].double() for i in range(0, vocab, 100000))
    check("d_hidden", host(dh), host(ref), BF16_REL_L2, None)
    tail = slice(vocab - 64, vocab)
    check("d_w", host(dw[tail]), host(dz[:, tail].T @ th.double()), BF16_REL_L2, None)


@pytest.mark.parametrize("types,rows", [(("bf16", "bf16"), 130), (("f32", "bf16"), 9), (("bf16", "bf16"), 3),
                                        (("f32", "f32"), 140), (("f32", "f32"), 7)])
def test_repeats_streams_and_neighbours(lib, types, rows):
    """The same bits on a second run, on another stream, in a captured graph that is replayed
    on new inputs, beside a second graph on the same workspace; memory behind the outputs
    stays as it was."""
    import torch
    vocab, dim = 3000, 200
    th, tw, h, w, t, g = problem(rows, vocab, dim, types)
    tt, tg = torch.from_numpy(t).cuda(), dev(g)
    ws = lib.xent_workspace(th.dtype, tw.dtype, rows, vocab, dim, grad_w=True)

    def call(out):
        lib.xent_forward(th, tw, tt, out[0][:rows], out[1][:rows], ws=ws)
        lib.xent_backward(th, tw, tt, out[1][:rows], tg, out[2][:rows], out[3][:vocab], ws=ws)

    def outputs():
        return [torch.full((n,) + s, 7.0, device="cuda", dtype=d) for n, s, d in
                ((rows + 3, (), torch.float32), (rows + 3, (), torch.float32), (rows + 3, (dim,), th.dtype),
                 (vocab + 3, (dim,), th.dtype))]

    first, second = outputs(), outputs()
    call(first)
    torch.cuda.synchronize()
    for out, n in zip(first, (rows, rows, rows, vocab)):
        assert bool((out[n:] == 7.0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(second)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    graphs = []
    for out in (third := outputs()), (fourth := outputs()):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(out)
        graphs.append(graph)
    th.copy_(th.roll(1, 0))
    fresh = outputs()
    call(fresh)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fresh, third))
    assert all(torch.equal(a, b) for a, b in zip(fresh, fourth))
    lib.workspace_status(ws)


def test_gradient_matches_differences_of_the_loss(lib):
    """The float32 gradient against central differences of the float32 loss along random directions."""
    import torch
    rows, vocab, dim = 40, 500, 96
    th, tw, _, _, t, g = problem(rows, vocab, dim, ("f32", "f32"))
    tt, tg = torch.from_numpy(t).cuda(), dev(g)
    loss, lse = lib.xent_forward(th, tw, tt)
    dh, dw = lib.xent_backward(th, tw, tt, lse, tg, grad_w=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    total = lambda h_, w_: float((lib.xent_forward(h_, w_, tt)[0].double() * tg.double()).sum())
    for x, dx, f in ((th, dh, lambda y: total(y, tw)), (tw, dw, lambda y: total(th, y))):
        d = torch.randn(x.shape, generator=gen, device="cuda")
        eps = 1e-2 / float(d.abs().max())
        along = float((dx.double() * d.double()).sum())
        diff = (f(x + eps * d) - f(x - eps * d)) / (2 * eps)
        # rounding of the loss: rows sqrt(40) x 6 x 2^-22 / eps ~ 4e-3; third derivative:
        # eps^2 |z''| z' ~ 1e-5 of a slope of |dx| ~ 10
        assert abs(along - diff) <= 1e-2 * max(1.0, float(dx.double().norm())), (along, diff)


def test_empty_and_refused(lib):
    import torch
    h, w = torch.zeros(0, 16, device="cuda"), torch.ones(5, 16, device="cuda")
    t, f = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, device="cuda")
    loss, lse = lib.xent_forward(h, w, t)
    assert loss.numel() == 0 and lse.numel() == 0
    dh, dw = lib.xent_backward(h, w, t, f, f, grad_w=True)
    assert dh.shape == (0, 16) and dw.shape == (5, 16) and not bool(dw.any())
    h = torch.zeros(3, 16, device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(lib.TlbError, match="float32 head"):
        lib.xent_forward(h, w, t)
    with pytest.raises(TypeError):
        lib.xent_forward(h, w.half(), t)
    with pytest.raises(TypeError, match="targets"):
        lib.xent_forward(h, w.bfloat16(), t.int())
    with pytest.raises(ValueError, match="targets"):
        lib.xent_forward(h, w.bfloat16(), t[:2])
    with pytest.raises(ValueError, match="contiguous"):
        lib.xent_forward(h, w.bfloat16().t().contiguous().t(), t)
    flat = torch.zeros(3 * 16 + 1, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(lib.TlbError, match="16-byte aligned"):
        lib.xent_forward(flat[1:].view(3, 16), w.bfloat16(), t)
    with pytest.raises(lib.TlbError, match="workspace"):
        lib.xent_forward(h, w.bfloat16(), t, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("types,rows,grad_w", [(("bf16", "bf16"), 3, True), (("bf16", "bf16"), 70, True),
                                               (("bf16", "bf16"), 300, False), (("f32", "bf16"), 10, True),
                                               (("f32", "f32"), 40, True)])
def test_gradient_in_place_of_the_hidden_rows(lib, types, rows, grad_w):
    """d_hidden may be hidden itself: the same bits, in one piece of the vocabulary or several."""
    import torch
    for vocab, dim in ((700, 96), (2100 if rows < 100 else 900000, 33)):
        th, tw, _, _, t, g = problem(rows, vocab, dim, types)
        tt, tg = torch.from_numpy(t).cuda(), dev(g)
        _, lse = lib.xent_forward(th, tw, tt)
        dh, dw = lib.xent_backward(th, tw, tt, lse, tg, grad_w=grad_w)
        same, dw2 = lib.xent_backward(th, tw, tt, lse, tg, d_hidden=th, grad_w=grad_w)
        assert same is th and torch.equal(th, dh)
        assert not grad_w or torch.equal(dw, dw2)


def test_what_is_allocated_belongs_to_the_given_stream(lib, monkeypatch):
    import torch
    th, tw, _, _, t, g = problem(20, 600, 64, ("bf16", "bf16"))
    tt, tg = torch.from_numpy(t).cuda(), dev(g)
    loss, lse = lib.xent_forward(th, tw, tt)
    dh, _ = lib.xent_backward(th, tw, tt, lse, tg)
    side, seen = torch.cuda.Stream(), []
    make = lib.api.xent_workspace

    def recorded(*args, **kw):
        seen.append(torch.cuda.current_stream())
        return make(*args, **kw)

    monkeypatch.setattr(lib.api, "xent_workspace", recorded)
    side.wait_stream(torch.cuda.current_stream())
    loss2, lse2 = lib.xent_forward(th, tw, tt, stream=side)
    dh2, _ = lib.xent_backward(th, tw, tt, lse2, tg, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert seen == [side, side]
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2) and torch.equal(dh, dh2)
