"""LayerNorm with residual, the linear with activation and their backward passes on tensors of more than 2^31 elements:
the first and last rows, and those on either side of the 2^31st element, against the 64-bit oracle.  Tolerances as in
test_gpu_act and test_gpu_add_layernorm, for the short contractions used here."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle.act import act_dgrad, linear_act
from tests import gpu_util as G
from tests.test_gpu_gated import BF, E23

pytestmark = pytest.mark.gpu
ROWS, COLS = 131_104, 16_400      # 2.15e9 elements; 2^31 lies in row 130 944
AT = [0, 1, 130_943, 130_944, 130_945, ROWS - 2, ROWS - 1]


def _f64(t):
    return t[AT].cpu().double().numpy()


def _random(rows, cols, seed, size=1.0):
    g = torch.Generator(device=G.DEV).manual_seed(seed)
    return torch.empty(rows, cols, dtype=torch.bfloat16, device=G.DEV).normal_(0.0, size, generator=g)


def test_layernorm():
    C = 16_384
    x, gamma, beta = _random(ROWS, C, 1), torch.linspace(0.5, 1.5, C, device=G.DEV), torch.linspace(-1, 1, C, device=G.DEV)
    y, mu, rs = torch.full_like(x, 7.0), torch.empty(ROWS, device=G.DEV), torch.empty(ROWS, device=G.DEV)
    q = torch.full((ROWS, C), 0x7F, dtype=torch.uint8, device=G.DEV)
    te.te_add_layernorm_fp8(x, gamma, beta, 1e-5, te.E4M3, G.scalar(16.0), q, y=y, mu=mu, rsigma=rs)
    torch.cuda.synchronize()
    v = _f64(x)
    m, r = v.mean(1, keepdims=True), 1 / np.sqrt(v.var(1, keepdims=True) + 1e-5)
    g64, b64 = gamma.cpu().double().numpy(), beta.cpu().double().numpy()
    want = (v - m) * r * g64 + b64
    # mean and variance: 2^14 terms, a few additions a lane and five butterflies each: well within 64 roundings
    slack = 64 * E23 * (np.abs(want) + np.abs(v) * r * g64 + 1)
    assert np.all(np.abs(_f64(y) - want) <= BF * (np.abs(want) + slack) + slack)
    got = q.view(torch.float8_e4m3fn)[AT].cpu().float().double().numpy() / 16
    top = np.clip(want, -28, 28)
    assert np.all(np.abs(got - top) <= 2.0 ** -4 * (np.abs(top) + slack) + slack + 2.0 ** -10 / 16)
    del q
    dx, dy = torch.full_like(x, 7.0), y
    dg, db = torch.empty(C, device=G.DEV), torch.empty(C, device=G.DEV)
    ws = torch.empty(te.te_layernorm_bwd_workspace_bytes(ROWS, C) // 4, device=G.DEV)
    te.te_layernorm_bwd(dy, x, gamma, mu, rs, dx, dg, db, ws)
    torch.cuda.synchronize()
    d, xh = _f64(dy), (v - m) * r
    p = d * g64
    want = r * (p - p.mean(1, keepdims=True) - xh * (p * xh).mean(1, keepdims=True))
    slack = 64 * E23 * r * (np.abs(p) + np.abs(p).mean(1, keepdims=True) + np.abs(xh) * np.abs(p * xh).mean(1, keepdims=True))
    assert np.all(np.abs(_f64(dx) - want) <= BF * (np.abs(want) + slack) + slack)
    total = torch.zeros(C, dtype=torch.float64, device=G.DEV)
    size = torch.zeros_like(total)
    for a in range(0, ROWS, 8192):
        part = dy[a:a + 8192].double()
        total += part.sum(0)
        size += part.abs().sum(0)
    # 131104 / 304 rows a partial sum, then 304 of them: under 1024 additions
    assert bool(((db.double() - total).abs() <= 1024 * 2.0 ** -24 * size).all())
    G.check_no_device_error()


def test_linear():
    K = 48
    x, w = _random(ROWS, K, 2), _random(COLS, K, 3, 0.2)
    bias = torch.linspace(-1, 1, COLS, device=G.DEV)
    z, y = (torch.full((ROWS, COLS), 7.0, dtype=torch.bfloat16, device=G.DEV) for _ in range(2))
    te.te_act_gemm_bf16(x, w, te.ACT_RELU, y=y, z=z, bias=bias)
    torch.cuda.synchronize()
    wv = w.cpu().double().numpy()
    y64, z64, _ = linear_act(_f64(x), wv, "relu", bias.cpu().double().numpy(), None)
    dz = (K + 4) * E23 * (np.abs(_f64(x)) @ np.abs(wv).T) + E23 * np.abs(z64)
    assert np.all(np.abs(_f64(z) - z64) <= BF * (np.abs(z64) + dz) + dz)
    assert np.all(np.abs(_f64(y) - y64) <= BF * (np.abs(y64) + dz) + dz)
    res = y     # in place
    before = _f64(res)
    te.te_act_gemm_bf16(x, w, te.ACT_NONE, y=y, residual=res)
    torch.cuda.synchronize()
    want = _f64(x) @ wv.T + before
    err = dz + E23 * np.abs(want)
    assert np.all(np.abs(_f64(y) - want) <= BF * (np.abs(want) + err) + err)
    # backward: dh = dy W2 with W2 [K, COLS]
    dy, w2 = _random(ROWS, K, 4), _random(K, COLS, 5, 0.2)
    d, db = y, torch.empty(COLS, device=G.DEV)
    ws = torch.empty(te.te_act_dbias_workspace_bytes(ROWS, COLS) // 4, device=G.DEV)
    te.te_act_bwd_bf16(x, w, w2, dy, z, te.ACT_RELU, d, db, ws)
    torch.cuda.synchronize()
    w2v, zs = w2.cpu().double().numpy(), _f64(z)
    want, _ = act_dgrad(_f64(dy), w2v, zs, "relu")
    slack = (K + 4) * E23 * (np.abs(_f64(dy)) @ np.abs(w2v))
    assert np.all(np.abs(_f64(d) - want) <= BF * (np.abs(want) + slack) + slack)
    total = torch.zeros(COLS, dtype=torch.float64, device=G.DEV)
    size = torch.zeros_like(total)
    for a in range(0, ROWS, 8192):
        part = d[a:a + 8192].double()
        total += part.sum(0)
        size += part.abs().sum(0)
    # dbias adds dz before its rounding: half a step of each, and under 256 additions (32 rows a part, 4097 parts: 5 + 129 + 5)
    assert bool(((db.double() - total).abs() <= (BF + 256 * 2.0 ** -24) * size * (1 + BF)).all())
    G.check_no_device_error()
