"""bf16 gradients of the linear-head cross entropy lose nothing of the targets' dz.

dz = g (p - onehot) is rounded to bf16 as an operand of the gradient products, and so are the
results, with relative errors of one size u (root mean square) each.  With logits near 0 every
p is about 1 / vocab, and a row's dz has a target's of size g beside vocab others that are
sqrt(vocab) (g / vocab) together.  Where only these are rounded, the squared error of either
gradient is u^2 (1 + 1 / vocab) of its squared size: at vocab >= 1000 it is that of the
result's own rounding but for 5e-4 (and a spread of p of exp(0.3^2); at 300 for 2e-3).  The
fp32 sums add 1e-5, 5e-5 of u's square.  So 1.02 times the rounding alone; with the targets' dz rounded
too it is sqrt(2).
"""
import numpy as np
import pytest

from tests.test_gpu_xent import dev

pytestmark = pytest.mark.gpu


def inputs(rows, vocab, dim, hot=0.0, seed=0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + vocab + seed)
    h = torch.randn(rows, dim, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(vocab, dim, generator=gen, device="cuda") * 0.3 / dim ** 0.5).bfloat16()
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    t[torch.rand(rows, generator=gen, device="cuda") < 0.1] = -1
    t[torch.rand(rows, generator=gen, device="cuda") < hot] = vocab // 2      # many rows with one target
    t[0], t[1], t[rows - 1] = 0, vocab - 1, vocab
    t[2], t[3] = 2 ** 40 + 5, -2 ** 32 + 5                   # no column, whatever their low bits say
    g = torch.rand(rows, generator=gen, device="cuda") + 0.5
    return h, w, t, g


def exact(h, w, t, lse, g):
    """(d_hidden, d_w) in float64."""
    import torch
    has = (t >= 0) & (t < len(w))
    dz = torch.exp(h.double() @ w.double().T - lse.double()[:, None])
    dz[torch.arange(len(t), device=t.device)[has], t[has]] -= 1.0
    dz *= (g.double() * has)[:, None]
    return dz @ w.double(), dz.T @ h.double()


def error(x, ref):
    return float((x.double() - ref).norm() / ref.norm())


SHAPES = [(65, 1000, 64, 0.0), (100, 1003, 136, 0.0), (128, 3000, 72, 0.5), (129, 3000, 130, 0.0), (300, 3001, 1001, 0.3),
          (777, 5000, 1000, 0.0), (1000, 20011, 328, 0.05), (300, 40000, 33, 0.0), (5000, 1000, 64, 0.0), (4100, 300, 520, 0.3),
          (20000, 2048, 40, 0.0), (2500, 9001, 264, 0.9)]


@pytest.mark.parametrize("rows,vocab,dim,hot", SHAPES)
def test_targets_are_not_rounded(lib, rows, vocab, dim, hot):
    import torch
    h, w, t, g = inputs(rows, vocab, dim, hot)
    _, lse = lib.xent_forward(h, w, t)
    dh, dw = lib.xent_backward(h, w, t, lse, g, grad_w=True)
    for name, got, ref in zip(("d_hidden", "d_w"), (dh, dw), exact(h, w, t, lse, g)):
        own = error(ref.bfloat16(), ref)                     # the rounding of the result alone
        assert error(got, ref) <= 1.02 * own, (name, error(got, ref) / own)


@pytest.mark.parametrize("rows,vocab,dim,hot", SHAPES)
def test_d_hidden_does_not_depend_on_d_w(lib, rows, vocab, dim, hot):
    import torch
    h, w, t, g = inputs(rows, vocab, dim, hot)
    _, lse = lib.xent_forward(h, w, t)
    both, _ = lib.xent_backward(h, w, t, lse, g, grad_w=True)
    alone, _ = lib.xent_backward(h, w, t, lse, g)
    assert torch.equal(both, alone)


def test_pieces_of_the_vocabulary(lib):
    """Two pieces (140000 rows leave room for 2048 columns of dz): targets in either."""
    import torch
    rows, vocab, dim = 140000, 4001, 40
    h, w, t, g = inputs(rows, vocab, dim)
    _, lse = lib.xent_forward(h, w, t)
    n0 = lib.launch_count()
    dh, dw = lib.xent_backward(h, w, t, lse, g, grad_w=True)
    assert lib.launch_names(n0).count("xent_dw") == 2
    for got, ref in zip((dh, dw), exact(h, w, t, lse, g)):
        assert error(got, ref) <= 1.02 * error(ref.bfloat16(), ref)


def test_one_target_for_all(lib):
    import torch
    rows, vocab, dim = 3000, 9001, 264
    h, w, t, g = inputs(rows, vocab, dim, hot=1.0)
    _, lse = lib.xent_forward(h, w, t)
    dh, dw = lib.xent_backward(h, w, t, lse, g, grad_w=True)
    v = vocab // 2
    rdw = exact(h, w, t, lse, g)[1][v]
    # 3000 products whose dz loses nothing: the result's rounding (half a step, 2^-8), and the fp32 sum's 1e-5
    # of the terms' absolute sum
    terms = (g.double()[:, None] * h.double().abs()).sum(0)
    assert bool(((dw[v].double() - rdw).abs() <= 2.0 ** -8 * rdw.abs() + 1e-5 * terms).all())
