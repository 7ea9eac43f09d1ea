"""Column sums over tensors of more than 2^31 elements, in whole numbers: LayerNorm's dgamma and dbeta and the linear's
dbias are compared for equality, so that a row left out, or added twice, shows.  (The sums stay below 2^24.)"""
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
ROWS = 131_104          # x 16384 and x 16400: 2^31 lies in rows 131 072 and 130 944


def _integers(rows, cols, lo, hi, seed):
    g = torch.Generator(device=G.DEV).manual_seed(seed)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=G.DEV)
    for a in range(0, rows, 16384):
        out[a:a + 16384] = torch.randint(lo, hi + 1, (min(16384, rows - a), cols), device=G.DEV, generator=g, dtype=torch.int8)
    return out


def test_layernorm_gradients():
    """mu = 0 and rsigma = 1, as a caller may give them: xhat is s itself."""
    C = 16_384
    dy, s = _integers(ROWS, C, 1, 3, 1), _integers(ROWS, C, -2, 3, 2)
    one, dx = torch.ones(C, device=G.DEV), torch.empty_like(s)
    dg, db = torch.full((C,), -1.0, device=G.DEV), torch.full((C,), -1.0, device=G.DEV)
    ws = torch.empty(te.te_layernorm_bwd_workspace_bytes(ROWS, C) // 4, device=G.DEV)
    te.te_layernorm_bwd(dy, s, one, torch.zeros(ROWS, device=G.DEV), torch.ones(ROWS, device=G.DEV), dx, dg, db, ws)
    torch.cuda.synchronize()
    want = torch.zeros(2, C, dtype=torch.float64, device=G.DEV)
    for a in range(0, ROWS, 8192):
        d, x = dy[a:a + 8192].float(), s[a:a + 8192].float()
        want[0] += (d * x).sum(0, dtype=torch.float64)
        want[1] += d.sum(0, dtype=torch.float64)
    assert torch.equal(dg.double(), want[0]) and torch.equal(db.double(), want[1])
    assert int(want.abs().max()) < 2 ** 24
    G.check_no_device_error()


def test_bias_gradient():
    F, N = 16_400, 16
    dy, w2 = _integers(ROWS, N, -2, 3, 3), _integers(N, F, -1, 1, 4)
    z, dz = _integers(ROWS, F, -1, 2, 5), torch.empty(ROWS, F, dtype=torch.bfloat16, device=G.DEV)
    db = torch.full((F,), -1.0, device=G.DEV)
    ws = torch.empty(te.te_act_dbias_workspace_bytes(ROWS, F) // 4, device=G.DEV)
    te.te_act_bwd_bf16(None, None, w2, dy, z, te.ACT_RELU, dz, db, ws)
    torch.cuda.synchronize()
    want, size = torch.zeros(F, dtype=torch.float64, device=G.DEV), torch.zeros(F, dtype=torch.float64, device=G.DEV)
    for a in range(0, ROWS, 8192):
        dh = (dy[a:a + 8192].float() @ w2.float()) * (z[a:a + 8192] > 0)
        assert torch.equal(dz[a:a + 8192].float(), dh)
        want += dh.sum(0, dtype=torch.float64)
        size += dh.abs().sum(0, dtype=torch.float64)
    assert torch.equal(db.double(), want)
    assert int(size.max()) < 2 ** 24 and bool((size > 0).all())
    G.check_no_device_error()
