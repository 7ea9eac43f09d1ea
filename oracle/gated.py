"""Gated feed-forward projections and their gradient.

Test infrastructure (see ``oracle/__init__``).

h = act(g) * u with g = x Wg^T and u = x Wu^T; act is SiLU, g / (1 + exp(-g)), or the tanh form of
GELU, g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))).  For y = h W2^T and dy = dL/dy:
  dh = dy W2,  dg = dh u act'(g),  du = dh act(g),  dx = dg Wg + du Wu,
  dWg = dg^T x,  dWu = du^T x
Plain fp64 definitions, pinned by closed forms, loops and central differences
(tests/test_oracle_gated).
"""
from __future__ import annotations

import numpy as np

C0, C1 = np.sqrt(2.0 / np.pi), 0.044715


def act(g, kind: str):
    g = np.asarray(g, np.float64)
    if kind == "silu":
        return g / (1.0 + np.exp(-g))
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-2.0 * C0 * (g + C1 * g ** 3)))     # 1/2 (1 + tanh t) = 1 / (1 + exp(-2 t))


def act_grad(g, kind: str):
    g = np.asarray(g, np.float64)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s * (1.0 - s)
    # 1 + tanh t loses its digits in 64 bits from t = -10 on; the logistic form keeps them
    z = 2.0 * C0 * (g + C1 * g ** 3)
    s, r = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    return s + g * s * r * 2.0 * C0 * (1.0 + 3.0 * C1 * g ** 2)


def gated(x, w, kind: str):
    """(h [T, F], g, u) of x [T, K] and w [2 F, K] (the gate's rows, then the up projection's)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    F = w.shape[0] // 2
    g, u = x @ w[:F].T, x @ w[F:].T
    return act(g, kind) * u, g, u


def gated_bwd(dy, w2, g, u, kind: str):
    """(dg, du) [T, F] from dy [T, N] and w2 [N, F]."""
    dh = np.asarray(dy, np.float64) @ np.asarray(w2, np.float64)
    return dh * u * act_grad(g, kind), dh * act(g, kind)
