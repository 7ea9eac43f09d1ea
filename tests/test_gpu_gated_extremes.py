"""The gated backward pass where the pre-activations are as large as bf16 holds: the activations' slopes are 1 and
0 there, and no product of an overflow with a zero."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G
from tests.test_gpu_gated import ACT, BF, E23, Operand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("actk", ["silu", "gelu"])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "mxfp8", "nvfp4"])
def test_saturated_gates(kind, actk):
    T, F, N = 40, 272, 64
    rng = np.random.default_rng(21)
    g = torch.tensor([30.0, 300.0, 1e10, 1e19, 2e19, 1e20, 3e38]).bfloat16()
    g = torch.cat([g, -g]).repeat(T * F // 14 + 1)[:T * F].view(T, F)
    u = torch.from_numpy(rng.standard_normal((T, F))).bfloat16()
    gu = torch.cat([g, u], 1).contiguous().to(G.DEV)
    d, w = Operand(rng.standard_normal((T, N)) * 1e-3, kind), None
    w2 = rng.standard_normal((N, F)) * 0.05
    dgu = torch.full_like(gu, 7.0)
    if kind == "bf16":
        w, x = Operand(w2, kind), torch.zeros(T, 16, dtype=torch.bfloat16, device=G.DEV)
        te.te_gated_bwd_bf16(x, torch.zeros(2 * F, 16, dtype=torch.bfloat16, device=G.DEV), w.q, d.q, gu, ACT[actk], dgu)
        w2v = w.v
    else:
        w = Operand(w2.T, kind)
        w2v = w.v.T
        if kind == "fp8":
            te.te_gated_dgrad_fp8(d.q, te.E4M3, w.q, te.E4M3, d.inv, w.inv, gu, ACT[actk], dgu)
        elif kind == "mxfp8":
            te.te_gated_dgrad_mxfp8(d.q, d.s, w.q, w.s, gu, ACT[actk], dgu)
        else:
            te.te_gated_dgrad_nvfp4(d.q, d.s, d.g, w.q, w.s, w.g, gu, ACT[actk], dgu)
    torch.cuda.synchronize()
    dh, S = d.v @ w2v, np.abs(d.v) @ np.abs(w2v) * (N + 4) * E23
    gv, uv = g.double().numpy(), u.double().numpy()
    on = gv > 0                                            # act(g) = g and its slope 1; otherwise 0 and 0, but for e^-30
    got = dgu.cpu().double().numpy()
    for part, want, size in ((got[:, :F], dh * uv * on, np.abs(uv) * on),
                             (got[:, F:], dh * np.where(on, gv, 0.0), np.where(on, gv, 0.0))):
        # (at g = -30: e^-30 of 30, below 3e-12 of it)
        tol = BF * (np.abs(want) + S * size) + S * size + np.where(on, 0.0, 1e-10 * (np.abs(dh) + S))
        tol += 8 * E23 * (np.abs(want) + S * size) + 1e-38
        assert np.all(np.abs(part - want) <= tol), (kind, actk, np.isnan(part).sum())
    G.check_no_device_error()
