"""The linear-head cross entropy in several pieces of the vocabulary where the head is packed:
a float32 head past 512 rows (three bf16 terms, 512 MB of them at most: 2 x 3 x 2560 bytes a
row of 2560 leave room for 34952), and a bf16 head whose rows are no multiple of 16 bytes.
Compared with float64 on the GPU; tolerances as in the operator's other tests.
"""
import numpy as np
import pytest

from tests.helpers import BF16_REL_L2, check, host

pytestmark = pytest.mark.gpu


def inputs(rows, vocab, dim, types, edges):
    """Hidden rows, head, targets (some without one, some around the pieces' edges), weights."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + vocab)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16}
    h = torch.randn(rows, dim, generator=gen, device="cuda").to(kind[types[0]])
    w = (torch.randn(vocab, dim, generator=gen, device="cuda") * (1.5 / dim ** 0.5)).to(kind[types[1]])
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    t[torch.rand(rows, generator=gen, device="cuda") < 0.2] = -1
    special = torch.tensor([0, vocab - 1, vocab] + [e + d for e in edges for d in (-1, 0)], device="cuda")[:rows]
    t[:len(special)] = special
    return h, w, t, torch.rand(rows, generator=gen, device="cuda") + 0.2


def exact(h, w, t, lse, g, step=20000):
    """(loss, lse, d_hidden, d_w) in float64, the gradients for the lse that is given."""
    import torch
    has = (t >= 0) & (t < len(w))
    wide = h.double()
    parts, at = [], torch.zeros(len(t), dtype=torch.float64, device="cuda")
    dh, dw = torch.zeros_like(wide), []
    for v in range(0, len(w), step):
        piece = w[v:v + step].double()
        z = wide @ piece.T
        here = has & (t >= v) & (t < v + step)
        parts.append(torch.logsumexp(z, 1))
        at[here] = z[here, t[here] - v]
        dz = torch.exp(z - lse.double()[:, None])
        dz[here, t[here] - v] -= 1.0
        dz *= (g.double() * has)[:, None]
        dh += dz @ piece
        dw.append(dz.T @ wide)
    rlse = torch.logsumexp(torch.stack(parts, 1), 1)
    return torch.where(has, rlse - at, torch.zeros_like(rlse)), rlse, dh, torch.cat(dw)


CASES = [(("f32", "f32"), 520, 36000, 2560, (18176, 18432)),       # two pieces in each direction
         (("f32", "f32"), 700, 11003, 8200, (5632,)),              # ... of other lengths
         (("bf16", "bf16"), 6, 300007, 1001, (150016, 150272)),    # bf16 rows of 2002 bytes
         (("bf16", "bf16"), 140, 300007, 1001, (150016,)),
         (("f32", "bf16"), 70, 300007, 1001, (150016,))]


@pytest.mark.parametrize("types,rows,vocab,dim,edges", CASES)
def test_packed_head_in_pieces(lib, types, rows, vocab, dim, edges):
    import torch
    h, w, t, g = inputs(rows, vocab, dim, types, edges)
    n0 = lib.launch_count()
    loss, lse = lib.xent_forward(h, w, t)
    n1 = lib.launch_count()
    dh, dw = lib.xent_backward(h, w, t, lse, g, grad_w=True)
    forward, backward = lib.launch_names(n0, n1), lib.launch_names(n1)
    pieces = forward.count("xent_stats")
    assert pieces >= 2 and forward.count("xent_pack") == pieces + 1 and forward.count("xent_join") == 1, forward
    assert backward.count("xent_grad") == backward.count("xent_dh") == backward.count("xent_dw") >= 2, backward
    assert not any(n.startswith("xent_token") for n in forward + backward)
    rloss, rlse, rdh, rdw = exact(h, w, t, lse, g)
    check("loss", host(loss), host(rloss))
    check("lse", host(lse), host(rlse))
    bar = (BF16_REL_L2, None) if types[0] == "bf16" else ()
    check("d_hidden", host(dh), host(rdh), *bar)
    check("d_w", host(dw), host(rdw), *bar)
    # the rows of each target, and those about the pieces' edges, by themselves
    for v in {int(x) for x in t[:3 + 2 * len(edges)].tolist()} & set(range(vocab)):
        near = slice(max(0, v - 8), v + 9)
        check("d_w near %d" % v, host(dw[near]), host(rdw[near]), *bar)
    only, none = lib.xent_backward(h, w, t, lse, g)
    assert none is None
    check("d_hidden alone", host(only), host(rdh), *bar)


def test_row_chunks_of_a_packed_head(lib):
    """The loss of more rows than one pass takes (16384), under a head in two pieces."""
    import torch
    rows, vocab, dim = 16390, 4099, 24000
    h, w, t, _ = inputs(rows, vocab, dim, ("f32", "f32"), (2048,))
    n0 = lib.launch_count()
    loss, lse = lib.xent_forward(h, w, t)
    names = lib.launch_names(n0)
    assert names.count("xent_stats") == 4 and names.count("xent_join") == 2, names
    for part in (slice(0, 200), slice(16300, rows)):
        z = h[part].double() @ w.double().T
        rlse = torch.logsumexp(z, 1)
        has = (t[part] >= 0) & (t[part] < vocab)
        at = z.gather(1, torch.where(has, t[part], torch.zeros_like(t[part]))[:, None])[:, 0]
        check("lse", host(lse[part]), host(rlse))
        check("loss", host(loss[part]), host(torch.where(has, rlse - at, torch.zeros_like(rlse))))
