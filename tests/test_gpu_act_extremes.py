"""The activations far out, in every form of the linear: from |z| = 200 on, SiLU, GELU and ReLU are z or zero and their
slopes one or zero, exactly, up to the largest bf16 (whose square and cube are not finite in fp32); from there down to
subnormal z within the tolerances of test_gpu_act.  One product each, so that z is exact."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle.act import act, act_grad
from tests import gpu_util as G
from tests.test_gpu_act import ACT, _sigmoid_error
from tests.test_gpu_act_forms import form
from tests.test_gpu_gated import BF, E23, Out

pytestmark = pytest.mark.gpu
BIG = torch.finfo(torch.bfloat16).max
FAR = [200.0, 1e4, 1e10, 1.8e19, 1.9e19, 1e25, 6.9e12, BIG]
NEAR = [0.0, 1e-38, 1e-30, 1e-10, 1e-3, 0.5, 1.0, 5.0, 12.0, 30.0]


def _columns(N):
    v = torch.tensor([s * x for x in FAR + NEAR for s in (1.0, -1.0)]).bfloat16()
    return v.repeat(-(-N // len(v)))[:N]


def _check(got, z, actk, want, slack):
    far = np.abs(z) >= 199
    assert np.array_equal(got[far], want[far].astype(np.float32)), actk
    err = slack[~far]
    assert np.all(np.abs(got - want)[~far] <= E23 / 2 * (np.abs(want[~far]) + err) + err + 2.0 ** -126), actk


@pytest.mark.parametrize("actk", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("T,K,N,what", [(1, 512, 512, "decode"), (24, 528, 20016, "stream"), (24, 4112, 528, "stream shared"),
                                        (100, 528, 20016, "stream"), (2080, 2080, 3344, "pair"), (2080, 8208, 272, "pair shared")])
def test_forward(T, K, N, what, actk):
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=G.DEV)
    x[:, K // 2] = 1.0
    w = torch.zeros(N, K, dtype=torch.bfloat16, device=G.DEV)
    col = _columns(N)
    w[:, K // 2] = col.to(G.DEV)
    y, y16, z = Out(T, N, dtype=torch.float32), Out(T, N), Out(T, N)

    def call(stream=None):
        te.te_act_gemm_bf16(x, w, ACT[actk], y=y.t, z=z.t, stream=stream)

    call()
    te.te_act_gemm_bf16(x, w, ACT[actk], y=y16.t)
    torch.cuda.synchronize()
    z64 = np.tile(col.double().numpy(), (T, 1))
    with np.errstate(all="ignore"):
        want = act(z64, actk)
    np.testing.assert_array_equal(z.np(), z64)
    _check(y.np(), z64, actk, want, _sigmoid_error(np.minimum(np.abs(z64), 30), actk) * np.abs(want))
    far = np.abs(z64) >= 199
    np.testing.assert_array_equal(y16.np()[far], want[far].astype(np.float32))
    assert form(call)[0] == what
    G.check_no_device_error()


@pytest.mark.parametrize("actk", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("T,F,N", [(33, 272, 16), (300, 2064, 528), (128, 512, 8208)])
def test_slopes(T, F, N, actk):
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device=G.DEV)
    dy[:, N // 2] = 1.0
    w2 = torch.ones(N, F, dtype=torch.bfloat16, device=G.DEV)
    col = _columns(F)
    z = col.to(G.DEV).repeat(T, 1).contiguous()
    dz, db = Out(T, F), torch.empty(F, device=G.DEV)
    ws = torch.empty(te.te_act_dbias_workspace_bytes(T, F) // 4, device=G.DEV)
    x = torch.zeros(T, 16, dtype=torch.bfloat16, device=G.DEV)
    te.te_act_bwd_bf16(x, torch.zeros(F, 16, dtype=torch.bfloat16, device=G.DEV), w2, dy, z, ACT[actk], dz.t, db, ws)
    torch.cuda.synchronize()
    z64 = col.double().numpy()
    with np.errstate(all="ignore"):
        want = act_grad(z64, actk)
    far = np.abs(z64) >= 199
    want[far] = z64[far] > 0
    # s + z s (1 - s) z': the sigmoid's error in both terms, as in test_gpu_act
    near = np.minimum(np.abs(z64), 30)
    slack = np.where(far, 0.0, 8 * (1 + near) * (_sigmoid_error(near, actk) + 4 * E23))
    got = dz.np()
    assert np.array_equal(got[:, far], np.tile(want[far], (T, 1)))
    assert np.all(np.abs(got - want) <= BF * (np.abs(want) + slack) + slack)
    assert np.all(np.abs(db.cpu().double().numpy() - T * want) <= T * slack + T * T * 2.0 ** -24)
    G.check_no_device_error()
