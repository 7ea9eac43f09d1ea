"""The linear with bias, activation and residual, and its gradient.

Test infrastructure (see ``oracle/__init__``).

z = x W^T + b, y = act(z) + residual; act is none, ReLU, or one of ``oracle.gated``.  For L with
dy = dL/dy of the linear after it, y2 = act(z) W2^T:
  dz = (dy W2) act'(z),  db = sum_t dz,  dx = dz W,  dW = dz^T x
Plain fp64 definitions, pinned by closed forms, loops and central differences
(tests/test_oracle_act).
"""
from __future__ import annotations

import numpy as np

from . import gated


def act(z, kind: str):
    z = np.asarray(z, np.float64)
    if kind == "none":
        return z
    if kind == "relu":
        return np.where(z > 0, z, np.where(np.isnan(z), z, 0.0))
    return gated.act(z, kind)


def act_grad(z, kind: str):
    z = np.asarray(z, np.float64)
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    return gated.act_grad(z, kind)


def linear_act(x, w, kind: str, bias=None, residual=None):
    """(y [T, N], z, act(z)) of x [T, K] and w [N, K]."""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    a = act(z, kind)
    return (a if residual is None else a + np.asarray(residual, np.float64)), z, a


def act_dgrad(dy, w2, z, kind: str):
    """(dz [T, F], db [F]) from dy [T, N], w2 [N, F] and z [T, F]."""
    dz = np.asarray(dy, np.float64) @ np.asarray(w2, np.float64)
    if kind != "none":
        dz = dz * act_grad(z, kind)
    return dz, dz.sum(axis=0)
