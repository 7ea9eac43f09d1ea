"""LayerNorm of the rows of X, the step before the QKV and MLP-up Fprop.

Test infrastructure (see ``oracle/__init__``).

y[r, c] = (x[r, c] - mu_r) * rsigma_r * gamma[c] + beta[c], with mu_r the mean of
row r, var_r its (biased) variance and rsigma_r = 1 / sqrt(var_r + eps): the
te.LayerNorm module that Transformer Engine fuses with the quantization of its
output ("Introduction to FP8 training using Transformer Engine", the module list
and fused kernels of the introduction and of section "Transformer Engine の使い方").
Plain fp64 definition; parity pinned by closed forms, invariances and loops
(tests/test_oracle_layernorm).
"""
from __future__ import annotations

import numpy as np


def layernorm(x, gamma, beta, eps: float):
    """(y [R, C], mu [R], rsigma [R]) in fp64."""
    x = np.asarray(x, dtype=np.float64)
    mu = x.mean(axis=1)
    var = ((x - mu[:, None]) ** 2).mean(axis=1)
    rsigma = 1.0 / np.sqrt(var + float(eps))
    y = (x - mu[:, None]) * rsigma[:, None] * np.asarray(gamma, np.float64)[None, :] + \
        np.asarray(beta, np.float64)[None, :]
    return y, mu, rsigma


def add_layernorm(x, gamma, beta, eps: float, residual=None):
    """(s [R, C], y [R, C], mu [R], rsigma [R]) in fp64, s = x + residual normalised."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    return (s, *layernorm(s, gamma, beta, eps))


def layernorm_bwd(dy, s, gamma, mu, rsigma, dres=None):
    """(ds [R, C], dgamma [C], dbeta [C]) in fp64, for L(y) with dy = dL/dy and a gradient dres that reaches s
    beside it:  ds = rsigma (p - mean(p) - xhat mean(p xhat)) + dres,  p = dy gamma, xhat = (s - mu) rsigma."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    rs = np.asarray(rsigma, np.float64)[:, None]
    xhat, p = (s - np.asarray(mu, np.float64)[:, None]) * rs, dy * np.asarray(gamma, np.float64)
    ds = rs * (p - p.mean(axis=1, keepdims=True) - xhat * (p * xhat).mean(axis=1, keepdims=True))
    if dres is not None:
        ds = ds + np.asarray(dres, np.float64)
    return ds, (dy * xhat).sum(axis=0), dy.sum(axis=0)
