"""Pins for oracle.rmsnorm: closed forms, loops, and central differences of the forward pass."""
import numpy as np

from oracle.rmsnorm import rmsnorm, rmsnorm_bwd

rng = np.random.default_rng(12)


def test_closed_forms():
    s, y, rs = rmsnorm([[3.0, 4.0]], [1.0, 2.0], 0.0)
    np.testing.assert_allclose(rs, [1 / np.sqrt(12.5)], rtol=1e-15)
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    s, y, rs = rmsnorm([[1.0, -2.0]], [1.0, 1.0], 1e-4, residual=[[-1.0, 2.0]])   # s = 0
    np.testing.assert_array_equal(s, 0.0)
    np.testing.assert_array_equal(y, 0.0)
    np.testing.assert_allclose(rs, [100.0], rtol=1e-15)


def test_loops():
    x, r, g = rng.standard_normal((3, 6)), rng.standard_normal((3, 6)), rng.standard_normal(6)
    s, y, rs = rmsnorm(x, g, 1e-5, r)
    for i in range(3):
        m = sum((x[i, j] + r[i, j]) ** 2 for j in range(6)) / 6
        for j in range(6):
            assert abs(y[i, j] - (x[i, j] + r[i, j]) / (m + 1e-5) ** 0.5 * g[j]) < 1e-13


def test_gradient_against_differences():
    x, r, g = rng.standard_normal((4, 10)), rng.standard_normal((4, 10)), rng.standard_normal(10)
    wy, ws = rng.standard_normal((4, 10)), rng.standard_normal((4, 10))   # L = <wy, y> + <ws, s>
    eps, h = 1e-3, 1e-5

    def loss(x, g):
        s, y, _ = rmsnorm(x, g, eps, r)
        return (wy * y).sum() + (ws * s).sum()

    s, _, rs = rmsnorm(x, g, eps, r)
    dx, dg = rmsnorm_bwd(wy, s, g, rs, ws)
    for i in range(4):
        for j in range(10):
            d = np.zeros_like(x)
            d[i, j] = h
            assert abs((loss(x + d, g) - loss(x - d, g)) / (2 * h) - dx[i, j]) < 1e-8
    for j in range(10):
        d = np.zeros_like(g)
        d[j] = h
        assert abs((loss(x, g + d) - loss(x, g - d)) / (2 * h) - dg[j]) < 1e-8
