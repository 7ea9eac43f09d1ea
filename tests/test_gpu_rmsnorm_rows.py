"""RMSNorm where every row group walks several rows, with an unequal last pass: the next row's loads, the
two slots of the row's sum behind one barrier, and the running amax.  Oracle and tolerances as in test_gpu_rmsnorm."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle.rmsnorm import rmsnorm
from tests import gpu_util as G
from tests.kernel_names import launched
from tests.test_gpu_rmsnorm import DT, E, EPS, FMAX, HALF, _bwd_check, _check_codes, _inputs, _np

pytestmark = pytest.mark.gpu

# (rows, cols, rows of a CTA): one to sixteen warps a row
WALKS = [(5003, 512, 8), (5003, 1024, 8), (2600, 1040, 4), (1501, 4096, 2), (701, 8192, 1), (331, 16384, 1)]


def _ctas(call):
    (ctas,) = [n for name, n in launched(call) if "rmsnorm_kernel" in name]
    return ctas


@pytest.mark.parametrize("rows,cols,per", WALKS)
@pytest.mark.parametrize("dtype,residual,fmt", [("bf16", True, "e4m3"), ("fp32", True, "e5m2"), ("bf16", False, "e5m2")])
def test_fp8(rows, cols, per, dtype, residual, fmt):
    x, r, gamma = _inputs(rows, cols, dtype, 11, residual)
    x[rows - 2, cols - 3] = 300.0                          # the largest y, in a late row
    if r is not None:
        r[rows - 2, cols - 3] = 0
    gamma[cols - 3] = 4.0
    s64, y64, rs64 = rmsnorm(_np(x), _np(gamma), EPS, None if r is None else _np(r))
    assert np.abs(y64).argmax() // cols == rows - 2
    scale = np.float32(FMAX[fmt] / (0.7 * np.abs(y64).max()))
    q, y = G.u8(rows, cols), torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=G.DEV)
    out, rs, amax, sc = torch.full_like(x, 7.0), torch.full((rows,), -1.0, device=G.DEV), G.scalar(-1.0), G.scalar(float(scale))

    def call(stream=None):
        te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3 if fmt == "e4m3" else te.E5M2, sc, q, residual=r, res_out=out, y=y,
                          rsigma=rs, amax_out=amax, stream=stream)

    call()
    torch.cuda.synchronize()
    assert np.all(np.abs(_np(out) - s64) <= (HALF[dtype] + E) * np.abs(s64))
    assert np.all(np.abs(_np(rs) - rs64) <= 40 * E * rs64)
    assert np.all(np.abs(_np(y) - y64) <= (HALF["bf16"] + 46 * E) * np.abs(y64))
    _check_codes(q.cpu().numpy(), y64 * float(scale), fmt)
    assert abs(amax.item() - np.abs(y64).max()) <= 44 * E * np.abs(y64).max()
    assert per * _ctas(call) < rows
    # a NaN in the last row stays there and reaches the amax
    want = q[:-1].clone()
    x[rows - 1, 5] = float("nan")
    call()
    torch.cuda.synchronize()
    assert np.isnan(amax.item()) and torch.equal(q[:-1], want) and bool(y[-1].isnan().all())
    G.check_no_device_error()


@pytest.mark.parametrize("rows,cols,per", WALKS)
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp32", True), ("fp32", False)])
def test_mxfp8(rows, cols, per, dtype, residual):
    cols -= cols % 32
    x, r, gamma = _inputs(rows, cols, dtype, 12, residual)
    s64, y64, _ = rmsnorm(_np(x), _np(gamma), EPS, None if r is None else _np(r))
    q, sr = G.u8(rows, cols), G.u8(te.te_scale_bytes(te.E8M0, rows, cols))
    out, y = torch.full_like(x, 7.0), torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=G.DEV)

    def call(stream=None):
        te.te_rmsnorm_mxfp8(x, gamma, EPS, q, sr, residual=r, res_out=out, y=y, stream=stream)

    call()
    torch.cuda.synchronize()
    raw = sr.cpu().numpy()
    s = te.te_scale_unswizzle(te.E8M0, rows, cols, raw).astype(np.int64)
    top = np.abs(y64).reshape(rows, cols // 32, 32).max(-1)
    lo, hi = (np.floor(np.log2(top * (1 + k * 46 * E))) - 8 + 127 for k in (-1, 1))
    assert np.all((s >= lo) & (s <= hi))
    _check_codes(q.cpu().numpy(), y64 * np.exp2(127.0 - np.repeat(s, 32, 1)), "e4m3")
    assert int(raw.astype(np.int64).sum()) == int(s.sum())               # padding is zero
    assert np.all(np.abs(_np(y) - y64) <= (HALF["bf16"] + 46 * E) * np.abs(y64))
    assert np.all(np.abs(_np(out) - s64) <= (HALF[dtype] + E) * np.abs(s64))
    assert per * _ctas(call) < rows
    G.check_no_device_error()


@pytest.mark.parametrize("rows,cols", [(5003, 512), (2600, 1040), (331, 8192), (331, 8208), (331, 16384)])
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp32", True), ("bf16", False)])
def test_backward(rows, cols, dtype, residual):
    _bwd_check(rows, cols, dtype, residual)
