"""A weight that is not finite, in the linear's backward pass: its own column of dz, and that column's sum, are not finite;
the rows past the last token, which are zero times it, add nothing to the sum, and every other column is what it would
be without it."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G
from tests.test_gpu_act import _bwd_inputs, _workspace, check_dz, dgrad
from tests.test_gpu_gated import Operand, Out

pytestmark = pytest.mark.gpu
SIZES = [(40, 176, 96), (1, 48, 32), (129, 272, 160), (300, 544, 96)]      # tokens, F, N: none fills its tiles
COL = 3


def _check(dz, db, d, w, z, actk, N, infinite):
    if infinite:       # positive products alone: + infinity; a zero times it would make it NaN
        assert np.isposinf(dz[:, COL]).all() and np.isposinf(db[COL])
    else:
        assert np.isnan(dz[:, COL]).all() and np.isnan(db[COL])
    rest = np.delete(np.arange(dz.shape[1]), COL)
    assert np.isfinite(dz[:, rest]).all() and np.isfinite(db[rest]).all()
    check_dz(dz[:, rest], db[rest], d, w[:, rest], z[:, rest], actk, N)


@pytest.mark.parametrize("T,F,N", SIZES)
@pytest.mark.parametrize("actk", ["relu", "gelu", "none"])
@pytest.mark.parametrize("kind", ["fp8", "mxfp8", "nvfp4"])
def test_dgrad(kind, actk, T, F, N):
    dy, w2, _ = _bwd_inputs(T, F, N)
    d, w = Operand(np.abs(dy) + 1e-4, kind, "e5m2"), Operand(w2.T, kind)
    z = torch.ones(T, F, dtype=torch.bfloat16, device=G.DEV)
    if kind == "fp8":
        w.q[COL] = 0x7F                                          # NaN, E4M3
    elif kind == "mxfp8":
        w.q[COL, 17] = 0x7F
    else:
        w.s[COL * 16] = 0x7F                                     # the block scale of the row's first 16 elements
    _, _, _, o, db = dgrad(kind, T, F, N, actk, ops=(d, w), z=z)
    _check(o.np(), db.cpu().double().numpy(), d.v, w.v.T, z.cpu().double().numpy(), actk, N, False)


@pytest.mark.parametrize("T,F,N", SIZES)
@pytest.mark.parametrize("actk", ["relu", "none"])
def test_an_infinite_weight_in_fp8(actk, T, F, N):
    dy, w2, _ = _bwd_inputs(T, F, N)
    d, w = Operand(np.abs(dy) + 1e-4, "fp8", "e5m2"), Operand(w2.T, "fp8", "e5m2")
    assert bool((d.q > 0).all())
    w.q[COL] = 1                                                 # the smallest positive number
    w.q[COL, N // 2] = 0x7C                                      # + infinity, E5M2
    z, dz, db = torch.ones(T, F, dtype=torch.bfloat16, device=G.DEV), Out(T, F), torch.full((F,), 7.0, device=G.DEV)
    te.te_act_dgrad_fp8(d.q, te.E5M2, w.q, te.E5M2, d.inv, w.inv, z, te.ACT_RELU if actk == "relu" else te.ACT_NONE, dz.t, db,
                        _workspace(T, F))
    torch.cuda.synchronize()
    G.check_no_device_error()
    _check(dz.np(), db.cpu().double().numpy(), d.v, w.v.T, np.ones((T, F)), actk, N, True)


@pytest.mark.parametrize("T,F,N", SIZES)
def test_an_infinite_weight_in_bf16(T, F, N):
    dy, w2, _ = _bwd_inputs(T, F, N)
    d, w = Operand(np.abs(dy) + 1e-4, "bf16"), Operand(w2, "bf16")
    w.q[:, COL] = 1.0
    w.q[N // 2, COL] = float("inf")
    z, dz, db = torch.ones(T, F, dtype=torch.bfloat16, device=G.DEV), Out(T, F), torch.full((F,), 7.0, device=G.DEV)
    te.te_act_bwd_bf16(None, None, w.q, d.q, z, te.ACT_RELU, dz.t, db, _workspace(T, F))
    torch.cuda.synchronize()
    G.check_no_device_error()
    _check(dz.np(), db.cpu().double().numpy(), d.v, w.v, np.ones((T, F)), "relu", N, True)
