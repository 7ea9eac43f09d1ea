"""Pins for oracle.gated: closed forms, loops, and central differences of the forward pass."""
import math

import numpy as np
import pytest

from oracle.gated import act, act_grad, gated, gated_bwd

rng = np.random.default_rng(13)


def test_closed_forms():
    np.testing.assert_allclose(act([0.0, math.log(3.0)], "silu"), [0.0, 0.75 * math.log(3.0)], rtol=1e-15)
    np.testing.assert_allclose(act_grad([0.0], "silu"), [0.5])
    np.testing.assert_allclose(act_grad([0.0], "gelu"), [0.5])
    np.testing.assert_allclose(act([40.0, -40.0], "gelu"), [40.0, 0.0], atol=1e-12)
    t = math.sqrt(2 / math.pi) * (1.5 + 0.044715 * 1.5 ** 3)
    np.testing.assert_allclose(act([1.5], "gelu"), [0.75 * (1 + math.tanh(t))], rtol=1e-15)
    # the tanh form stays within 5e-4 of the exact GELU g Phi(g)
    g = np.linspace(-6, 6, 241)
    phi = np.array([0.5 * (1 + math.erf(v / math.sqrt(2))) for v in g])
    assert np.abs(act(g, "gelu") - g * phi).max() < 5e-4


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_loops(kind):
    x, w = rng.standard_normal((3, 5)), rng.standard_normal((8, 5))
    h, g, u = gated(x, w, kind)
    for t in range(3):
        for f in range(4):
            gv = sum(x[t, k] * w[f, k] for k in range(5))
            uv = sum(x[t, k] * w[4 + f, k] for k in range(5))
            a = gv / (1 + math.exp(-gv)) if kind == "silu" else \
                gv / (1 + math.exp(-2 * math.sqrt(2 / math.pi) * (gv + 0.044715 * gv ** 3)))
            assert abs(h[t, f] - a * uv) < 1e-12 and abs(g[t, f] - gv) < 1e-13 and abs(u[t, f] - uv) < 1e-13


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient_against_differences(kind):
    x, w, w2 = rng.standard_normal((3, 5)), rng.standard_normal((8, 5)), rng.standard_normal((6, 4))
    dy, d = rng.standard_normal((3, 6)), 1e-5

    def loss(x, w):
        return (dy * (gated(x, w, kind)[0] @ w2.T)).sum()

    _, g, u = gated(x, w, kind)
    dgu = np.concatenate(gated_bwd(dy, w2, g, u, kind), 1)
    dx, dw = dgu @ w, dgu.T @ x
    for a, grad in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += d
            dn[i] -= d
            num = (loss(up, w) - loss(dn, w)) if a is x else (loss(x, up) - loss(x, dn))
            assert abs(num / (2 * d) - grad[i]) < 1e-7
