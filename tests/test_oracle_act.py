"""Pins for oracle.act and the new half of oracle.layernorm: closed forms, loops, central differences."""
import numpy as np
import pytest

from oracle.act import act, act_dgrad, act_grad, linear_act
from oracle.layernorm import add_layernorm, layernorm_bwd

rng = np.random.default_rng(31)


def test_activations():
    z = np.array([-2.0, -0.0, 0.0, 3.0, np.nan])
    np.testing.assert_array_equal(act(z, "relu"), [0.0, 0.0, 0.0, 3.0, np.nan])
    np.testing.assert_array_equal(act_grad(z[:4], "relu"), [0.0, 0.0, 0.0, 1.0])
    np.testing.assert_array_equal(act(z[:4], "none"), z[:4])
    np.testing.assert_array_equal(act_grad(z[:4], "none"), 1.0)


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
def test_linear_loops(kind):
    x, w, b, r = (rng.standard_normal(s) for s in ((3, 5), (4, 5), (4,), (3, 4)))
    y, z, a = linear_act(x, w, kind, b, r)
    for t in range(3):
        for n in range(4):
            v = sum(x[t, k] * w[n, k] for k in range(5)) + b[n]
            assert abs(z[t, n] - v) < 1e-13 and abs(y[t, n] - float(act(v, kind)) - r[t, n]) < 1e-13
    np.testing.assert_array_equal(linear_act(x, w, kind)[0], act(x @ w.T, kind))


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
def test_linear_gradient_against_differences(kind):
    x, w, b, w2, dy = (rng.standard_normal(s) for s in ((3, 5), (4, 5), (4,), (6, 4), (3, 6)))
    h = 1e-6

    def loss(x, w, b):
        return (dy * (linear_act(x, w, kind, b)[0] @ w2.T)).sum()

    z = linear_act(x, w, kind, b)[1]
    dz, db = act_dgrad(dy, w2, z, kind)
    for p, g in ((0, dz @ w), (1, dz.T @ x), (2, db)):
        at = [x, w, b]
        for i in np.ndindex(*at[p].shape):
            d = np.zeros_like(at[p])
            d[i] = h
            up, down = list(at), list(at)
            up[p], down[p] = at[p] + d, at[p] - d
            assert abs((loss(*up) - loss(*down)) / (2 * h) - g[i]) < 1e-7


def test_layernorm_gradient_against_differences():
    x, r = rng.standard_normal((4, 10)), rng.standard_normal((4, 10)) + 2.0
    g, b = rng.standard_normal(10), rng.standard_normal(10)
    wy, ws = rng.standard_normal((4, 10)), rng.standard_normal((4, 10))   # L = <wy, y> + <ws, s>
    eps, h = 1e-3, 1e-5

    def loss(x, g, b):
        s, y, _, _ = add_layernorm(x, g, b, eps, r)
        return (wy * y).sum() + (ws * s).sum()

    s, _, mu, rs = add_layernorm(x, g, b, eps, r)
    np.testing.assert_array_equal(s, x + r)
    grads = layernorm_bwd(wy, s, g, mu, rs, ws)
    at = [x, g, b]
    for p in range(3):
        for i in np.ndindex(*at[p].shape):
            d = np.zeros_like(at[p])
            d[i] = h
            up, down = list(at), list(at)
            up[p], down[p] = at[p] + d, at[p] - d
            assert abs((loss(*up) - loss(*down)) / (2 * h) - grads[p][i]) < 1e-8


def test_layernorm_closed_forms():
    s, y, mu, rs = add_layernorm([[1.0, 2.0]], [1.0, 3.0], [0.0, 1.0], 0.0, [[1.0, 2.0]])
    np.testing.assert_array_equal(s, [[2.0, 4.0]])
    np.testing.assert_allclose(y, [[-1.0, 4.0]], rtol=1e-15)
    np.testing.assert_allclose((mu, rs), [[3.0], [1.0]], rtol=1e-15)
    # a gradient that is the same in every column of xhat's plane carries nothing
    ds, dg, db = layernorm_bwd([[5.0, 5.0]], s, [1.0, 1.0], mu, rs)
    np.testing.assert_allclose(ds, 0.0, atol=1e-15)
    np.testing.assert_allclose((dg, db), [[-5.0, 5.0], [5.0, 5.0]])
