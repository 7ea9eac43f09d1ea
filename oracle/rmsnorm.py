"""Root-mean-square norm of the rows with the residual's addition, and its gradient.

Test infrastructure (see ``oracle/__init__``).

s = x + residual, rsigma_r = 1 / sqrt(mean_c s[r, c]^2 + eps), y = s * rsigma * gamma.
For L(y) with dy = dL/dy and a gradient dres that reaches s beside it:
  dL/ds[r, c]   = rsigma (p - xhat mean_c(p xhat)) + dres,  p = dy gamma, xhat = s rsigma
  dL/dgamma[c]  = sum_r dy[r, c] xhat[r, c]
Plain fp64 definitions, pinned by closed forms, loops and central differences
(tests/test_oracle_rmsnorm).
"""
from __future__ import annotations

import numpy as np


def rmsnorm(x, gamma, eps: float, residual=None):
    """(s [R, C], y [R, C], rsigma [R]) in fp64."""
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    rsigma = 1.0 / np.sqrt((s ** 2).mean(axis=1) + float(eps))
    return s, s * rsigma[:, None] * np.asarray(gamma, np.float64), rsigma


def rmsnorm_bwd(dy, s, gamma, rsigma, dres=None):
    """(ds [R, C], dgamma [C]) in fp64."""
    dy, s = np.asarray(dy, np.float64), np.asarray(s, np.float64)
    rs = np.asarray(rsigma, np.float64)[:, None]
    xhat, p = s * rs, dy * np.asarray(gamma, np.float64)
    ds = rs * (p - xhat * (p * xhat).mean(axis=1, keepdims=True))
    if dres is not None:
        ds = ds + np.asarray(dres, np.float64)
    return ds, (dy * xhat).sum(axis=0)
