"""Pins of the oracle's linear-head cross entropy: central differences of the loss, closed
forms, and rows without a target."""
import numpy as np
import pytest

from oracle import ops


def problem(rows, vocab, dim, seed=0):
    rs = np.random.default_rng(seed)
    t = rs.integers(0, vocab, rows)
    return rs.normal(size=(rows, dim)), rs.normal(0, 0.7, (vocab, dim)), t, rs.uniform(0.2, 1.5, rows)


@pytest.mark.parametrize("rows,vocab,dim", [(1, 2, 1), (3, 7, 5), (4, 11, 6)])
def test_gradients_match_finite_differences(rows, vocab, dim):
    h, w, t, g = problem(rows, vocab, dim)
    if rows > 1:
        t[1] = -1
    total = lambda h_, w_: float(np.sum(g * ops.xent_forward(h_, w_, t)[0]))
    dh, dw = ops.xent_backward(h, w, t, ops.xent_forward(h, w, t)[1], g)
    eps = 1e-6
    for x, dx, f in ((h, dh, lambda y: total(y, w)), (w, dw, lambda y: total(h, y))):
        for i in np.ndindex(x.shape):
            up, down = x.copy(), x.copy()
            up[i] += eps
            down[i] -= eps
            # central difference: eps^2 f'''/6 ~ 1e-12 plus rounding 1e-16 |f| / eps ~ 1e-9
            assert abs((f(up) - f(down)) / (2 * eps) - dx[i]) < 1e-7


def test_closed_forms():
    h, w = np.zeros((2, 3)), np.ones((8, 3))
    loss, lse = ops.xent_forward(h, w, [0, 7])
    assert np.allclose(lse, np.log(8)) and np.allclose(loss, np.log(8))     # equal logits
    dz = ops.xent_dlogits(h, w, [0, 7], lse, np.ones(2))
    assert np.allclose(dz.sum(1), 0) and np.allclose(dz[0, 0], 1 / 8 - 1) and np.allclose(dz[0, 1:], 1 / 8)
    loss, lse = ops.xent_forward(np.array([[1000.0]]), np.array([[1.0], [-1.0]]), [0])
    assert loss[0] == 0.0 and lse[0] == 1000.0                              # no overflow


def test_rows_without_a_target_add_nothing():
    h, w, t, g = problem(5, 9, 4)
    t[[1, 3]] = -100, 9
    loss, lse = ops.xent_forward(h, w, t)
    assert loss[1] == 0 and loss[3] == 0 and np.all(np.isfinite(lse))
    dh, dw = ops.xent_backward(h, w, t, lse, g)
    assert np.all(dh[[1, 3]] == 0)
    keep = [0, 2, 4]
    dh2, dw2 = ops.xent_backward(h[keep], w, t[keep], lse[keep], g[keep])
    assert np.allclose(dh[keep], dh2) and np.allclose(dw, dw2)
