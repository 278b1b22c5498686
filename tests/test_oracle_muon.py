"""Pins of the oracle's Muon step: the matrix recurrence, invariances and special cases."""
import numpy as np
import pytest

from oracle import ops

COEF = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (7, 3), (5, 5)])
def test_newton_schulz_is_the_matrix_recurrence(shape):
    x = np.random.default_rng(0).normal(size=shape)
    x /= np.linalg.norm(x)
    y = x
    for _ in range(5):
        gram = y @ y.T
        y = COEF[0] * y + COEF[1] * gram @ y + COEF[2] * gram @ gram @ y
    assert np.allclose(ops.newton_schulz(x, COEF, 5), y, rtol=0, atol=1e-12)


def test_newton_schulz_orthogonalises():
    # with the convergent coefficients (15, -10, 3) / 8 the singular values go to 1
    x = np.random.default_rng(1).normal(size=(4, 9))
    y = ops.newton_schulz(x / np.linalg.norm(x), (15 / 8, -10 / 8, 3 / 8), 40)
    assert np.allclose(y @ y.T, np.eye(4), atol=1e-12)
    q, _ = np.linalg.qr(np.random.default_rng(2).normal(size=(4, 4)))
    assert np.allclose(ops.newton_schulz(q @ x, COEF, 3), q @ ops.newton_schulz(x, COEF, 3))


def test_muon_step():
    rs = np.random.default_rng(3)
    p, g, m = (rs.normal(size=(4, 6)) for _ in range(3))
    p1, m1 = ops.muon(p, g, m, 0.1, 0.9, 0.5, 1e-7, COEF, 5, False, 2.0)
    assert np.allclose(m1, 0.9 * m + g)
    assert np.allclose(p1, p - 0.05 * p - 0.2 * ops.newton_schulz(m1 / np.linalg.norm(m1), COEF, 5), atol=1e-6)
    p2, m2 = ops.muon(p, g, m, 0.1, 0.9, 0.5, 1e-7, COEF, 5, True, 2.0)
    assert np.allclose(m2, m1) and not np.allclose(p2, p1)
    # the direction does not depend on the gradient's size
    a, _ = ops.muon(0 * p, g, 0 * m, 1.0, 0.9, 0.0, 0.0, COEF, 5, True, 1.0)
    b, _ = ops.muon(0 * p, 100 * g, 0 * m, 1.0, 0.9, 0.0, 0.0, COEF, 5, True, 1.0)
    assert np.allclose(a, b)
    z, mz = ops.muon(p, 0 * g, 0 * m, 0.1, 0.9, 0.5, 0.0, COEF, 5, True, 1.0)
    assert np.allclose(z, 0.95 * p) and not mz.any()
