"""RMSNorm with the residual's addition, its 8-bit outputs and its gradient, against the 64-bit oracle.

Tolerances count roundings.  E = 2^-24 is half a step of fp32, 2^-8 of bf16, 2^-4 of E4M3 and
2^-3 of E5M2 (relative).  A row's sum of squares is built from at most 32 terms per lane pair,
a 5-step butterfly and 16 warps' sums, all of one sign: at most 64 E relative, so rsigma (the
square root halves it; division, addition of eps, root and reciprocal add 4) is within 40 E and
y = (s rsigma) gamma, with s itself one rounding of x + residual, within 44 E before its own
rounding.  Where x and residual cancel, s is exact or off by E |s| all the same (one rounding).
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle import formats as F
from oracle.rmsnorm import rmsnorm, rmsnorm_bwd
from tests import gpu_util as G

E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": E, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
SMALL = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}         # half a step of the subnormals
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-5


def _inputs(rows, cols, dtype, seed=0, residual=True):
    g = torch.Generator().manual_seed(seed + 7 * rows + cols)
    x = torch.randn(rows, cols, generator=g)
    r = torch.randn(rows, cols, generator=g) * (1 + 30 * (torch.rand(cols, generator=g) < 0.02))
    gamma = 1 + 0.2 * torch.randn(cols, generator=g)
    return (x.to(DT[dtype]).to(G.DEV), r.to(DT[dtype]).to(G.DEV) if residual else None, gamma.to(G.DEV))


def _np(t):
    return t.detach().cpu().double().numpy()


def _check_codes(q, ideal, fmt, ulps=46):
    """Codes against the ideal values: half a step of the format beside the fp32 error."""
    got = F.decode(q, fmt).astype(np.float64)
    v = np.clip(ideal, -FMAX[fmt], FMAX[fmt])
    tol = np.maximum(HALF[fmt] * np.abs(v), SMALL[fmt]) + ulps * E * np.abs(v)
    assert np.all(np.abs(got - v) <= tol), float(np.max(np.abs(got - v) / tol))


SHAPES = [(1, 16), (1, 4096), (3, 48), (17, 1024), (9, 1040), (33, 2048), (5, 2064), (130, 4096), (7, 5120),
          (20, 8192), (3, 8208), (2, 16384), (1300, 768)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,residual,fmt", [("bf16", True, "e4m3"), ("fp32", True, "e5m2"), ("bf16", False, "e5m2"),
                                                ("fp32", False, "e4m3")])
def test_fp8(rows, cols, dtype, residual, fmt):
    x, r, gamma = _inputs(rows, cols, dtype, residual=residual)
    s64, y64, rs64 = rmsnorm(_np(x), _np(gamma), EPS, None if r is None else _np(r))
    scale = np.float32(FMAX[fmt] / (0.7 * np.abs(y64).max()))            # some values saturate
    q, y = G.u8(rows, cols), torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=G.DEV)
    out, rs = torch.full_like(x, 7.0), torch.full((rows,), -1.0, device=G.DEV)
    amax, inv = G.scalar(-1.0), G.scalar(-1.0)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3 if fmt == "e4m3" else te.E5M2, G.scalar(float(scale)), q, residual=r,
                      res_out=out, y=y, rsigma=rs, amax_out=amax, scale_inv_out=inv)
    torch.cuda.synchronize()
    assert np.all(np.abs(_np(out) - s64) <= (HALF[dtype] + E) * np.abs(s64))
    assert np.all(np.abs(_np(rs) - rs64) <= 40 * E * rs64)
    assert np.all(np.abs(_np(y) - y64) <= (HALF["bf16"] + 46 * E) * np.abs(y64))
    _check_codes(q.cpu().numpy(), y64 * float(scale), fmt)
    assert abs(amax.item() - np.abs(y64).max()) <= 44 * E * np.abs(y64).max()
    assert np.float32(inv.item()) == np.float32(1.0) / scale
    G.check_no_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (127, 160), (129, 1024), (40, 1056), (300, 4096),
                                       (5, 8224), (2, 16384)])
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp32", False)])
def test_mxfp8(rows, cols, dtype, residual):
    x, r, gamma = _inputs(rows, cols, dtype, 1, residual)
    s64, y64, rs64 = rmsnorm(_np(x), _np(gamma), EPS, None if r is None else _np(r))
    q, sr = G.u8(rows, cols), G.u8(te.te_scale_bytes(te.E8M0, rows, cols))
    out, y = torch.full_like(x, 7.0), torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=G.DEV)
    te.te_rmsnorm_mxfp8(x, gamma, EPS, q, sr, residual=r, res_out=out, y=y)
    torch.cuda.synchronize()
    raw = sr.cpu().numpy()
    s = te.te_scale_unswizzle(te.E8M0, rows, cols, raw).astype(np.int64)
    # the shared exponent, where the block's maximum may be off by 44 E either way
    top = np.abs(y64).reshape(rows, cols // 32, 32).max(-1)
    lo = np.floor(np.log2(top * (1 - 46 * E))) - 8 + 127
    hi = np.floor(np.log2(top * (1 + 46 * E))) - 8 + 127
    assert np.all((s >= lo) & (s <= hi))
    ideal = y64 * np.exp2(127.0 - np.repeat(s, 32, 1))
    _check_codes(q.cpu().numpy(), ideal, "e4m3")
    assert int(raw.astype(np.int64).sum()) == int(s.sum())               # padding is zero
    assert np.all(np.abs(_np(y) - y64) <= (HALF["bf16"] + 46 * E) * np.abs(y64))
    assert np.all(np.abs(_np(out) - s64) <= (HALF[dtype] + E) * np.abs(s64))
    G.check_no_device_error()


@pytest.mark.gpu
def test_optional_outputs_and_in_place():
    x, r, gamma = _inputs(40, 1024, "bf16", 2)
    y, y2, q = torch.empty_like(x), torch.empty_like(x), G.u8(40, 1024)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, residual=r, y=y)               # bf16 only: no scale needed
    out = torch.empty_like(x)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, G.scalar(3.0), q, residual=r, res_out=out)
    want_q = q.clone()
    for target in ("x", "r"):
        a, b = x.clone(), r.clone()
        q.zero_()
        te.te_rmsnorm_fp8(a, gamma, EPS, te.E4M3, G.scalar(3.0), q, residual=b, res_out=a if target == "x" else b, y=y2)
        torch.cuda.synchronize()
        assert torch.equal(a if target == "x" else b, out)
        assert torch.equal(q, want_q) and torch.equal(y, y2)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, G.scalar(3.0), q, y=x)         # y over x, no residual
    want = torch.empty_like(x)
    x2, _, _ = _inputs(40, 1024, "bf16", 2)
    te.te_rmsnorm_fp8(x2, gamma, EPS, te.E4M3, y=want)
    torch.cuda.synchronize()
    assert torch.equal(x, want)


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
def test_special_values(mx):
    """A zero row stays zero, a row of the largest values, infinities and NaN stay in their rows;
    the amax does not lose a NaN."""
    x, _, gamma = _inputs(6, 256, "fp32", 3)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e-30
    q, y = G.u8(6, 256), torch.empty(6, 256, dtype=torch.bfloat16, device=G.DEV)
    amax, rs = G.scalar(), torch.empty(6, device=G.DEV)
    if mx:
        s = G.u8(te.te_scale_bytes(te.E8M0, 6, 256))
        te.te_rmsnorm_mxfp8(x, gamma, EPS, q, s, y=y, rsigma=rs)
    else:
        te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, G.scalar(10.0), q, y=y, rsigma=rs, amax_out=amax)
    torch.cuda.synchronize()
    yn = y.float().cpu().numpy()
    _, y64, rs64 = rmsnorm(_np(x)[[0, 1, 4, 5]], _np(gamma), EPS)
    assert np.all(np.abs(yn[[0, 1, 4, 5]] - y64) <= (HALF["bf16"] + 46 * E) * np.abs(y64))
    assert not q[1].any() and np.all(yn[1] == 0)
    assert np.isnan(yn[2]).all() and rs.isnan().tolist() == [False, False, True, False, False, False]
    assert np.isnan(yn[3, 7]) and np.all(yn[3, :7] == 0)                  # rsigma = 1 / inf
    if mx:
        assert not te.te_scale_unswizzle(te.E8M0, 6, 256, s.cpu().numpy())[1].any()
    else:
        assert np.isnan(amax.item())


@pytest.mark.gpu
def test_no_rows():
    x, gamma = torch.empty(0, 64, dtype=torch.bfloat16, device=G.DEV), torch.ones(64, device=G.DEV)
    with pytest.raises(TypeError):        # a required tensor is missing
        te.te_rmsnorm_bwd(None, x, gamma, torch.empty(0, device=G.DEV), x, gamma, x)
    amax, inv = G.scalar(-1.0), G.scalar(-1.0)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, G.scalar(4.0), torch.empty(0, 64, dtype=torch.uint8, device=G.DEV),
                      amax_out=amax, scale_inv_out=inv)
    dgamma = torch.full((64,), 3.0, device=G.DEV)
    te.te_rmsnorm_bwd(x, x, gamma, torch.empty(0, device=G.DEV), x.clone(), dgamma, torch.empty(0, device=G.DEV))
    torch.cuda.synchronize()
    assert amax.item() == 0 and inv.item() == 0.25 and not dgamma.any()


def _bwd_check(rows, cols, dtype, residual, seed=4):
    x, _, gamma = _inputs(rows, cols, dtype, seed)
    g = torch.Generator().manual_seed(seed)
    dy = (torch.randn(rows, cols, generator=g) * 1e-3).bfloat16().to(G.DEV)
    dres = (torch.randn(rows, cols, generator=g) * 1e-3).to(DT[dtype]).to(G.DEV) if residual else None
    rs = torch.rsqrt(x.double().square().mean(1) + EPS).float()
    dx, dgamma = torch.full_like(x, 7.0), torch.full((cols,), 7.0, device=G.DEV)
    ws = torch.full((te.te_rmsnorm_bwd_workspace_bytes(rows, cols) // 4,), float("nan"), device=G.DEV)
    te.te_rmsnorm_bwd(dy, x, gamma, rs, dx, dgamma, ws, dres=dres)
    torch.cuda.synchronize()
    ds64, dg64 = rmsnorm_bwd(_np(dy), _np(x), _np(gamma), _np(rs), None if dres is None else _np(dres))
    # per element: p and xhat (2 roundings each), their mean (64 E of its absolute terms), two fused steps
    xhat = np.abs(_np(x)) * _np(rs)[:, None]
    p = np.abs(_np(dy) * _np(gamma))
    size = _np(rs)[:, None] * (p + xhat * (p * xhat).mean(1, keepdims=True))
    tol = 72 * E * size + (HALF[dtype] + E) * (np.abs(ds64) + 72 * E * size)
    assert np.all(np.abs(_np(dx) - ds64) <= tol), float(np.max(np.abs(_np(dx) - ds64) / tol))
    tol = (rows + 4) * E * (np.abs(_np(dy)) * xhat).sum(0)
    assert np.all(np.abs(_np(dgamma) - dg64) <= tol)
    G.check_no_device_error()
    return dy, x, gamma, rs, dres, dx, dgamma


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 4096), (700, 2048)])
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp32", True), ("bf16", False)])
def test_backward(rows, cols, dtype, residual):
    _bwd_check(rows, cols, dtype, residual)


@pytest.mark.gpu
def test_backward_in_place_and_repeatable():
    dy, x, gamma, rs, dres, dx, dgamma = _bwd_check(900, 1024, "bf16", True)
    ws = torch.empty(te.te_rmsnorm_bwd_workspace_bytes(900, 1024) // 4, device=G.DEV)
    for _ in range(2):
        for target in (dres.clone(), x.clone()):
            dg = torch.empty_like(dgamma)
            alias = target if target is not None else None
            same = torch.equal(alias, dres)
            te.te_rmsnorm_bwd(dy, x if same else alias, gamma, rs, alias, dg, ws, dres=alias if same else dres)
            torch.cuda.synchronize()
            assert torch.equal(alias, dx) and torch.equal(dg, dgamma)


@pytest.mark.gpu
def test_other_stream_and_graph():
    x, r, gamma = _inputs(600, 1024, "bf16", 5)
    q, q2, amax, amax2 = G.u8(600, 1024), G.u8(600, 1024), G.scalar(), G.scalar()
    sc = G.scalar(20.0)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, sc, q, residual=r, amax_out=amax)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, sc, q2, residual=r, amax_out=amax2, stream=side)
    side.synchronize()
    assert torch.equal(q, q2) and torch.equal(amax, amax2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, sc, q2, residual=r, amax_out=amax2)
    x.mul_(0.5)
    te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, sc, q, residual=r, amax_out=amax)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(amax, amax2)


@pytest.mark.gpu
def test_backward_in_a_graph():
    """The sums of dgamma start while the rows' kernel drains, eagerly and in a graph: the same bits."""
    dy, x, gamma, rs, dres, dx, dgamma = _bwd_check(2000, 768, "bf16", True)
    ws = torch.full((te.te_rmsnorm_bwd_workspace_bytes(2000, 768) // 4,), float("nan"), device=G.DEV)
    dx2, dg2 = torch.empty_like(dx), torch.empty_like(dgamma)
    for _ in range(20):
        te.te_rmsnorm_bwd(dy, x, gamma, rs, dx2, dg2, ws, dres=dres)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dgamma, dg2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            te.te_rmsnorm_bwd(dy, x, gamma, rs, dx2, dg2, ws, dres=dres)
        dg3 = dg2.clone()
    for _ in range(3):
        dg2.zero_()
        ws.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dgamma, dg3) and torch.equal(dx, dx2)


# ---- refusals: nothing reaches the GPU --------------------------------------------------------

def test_wrapper_refusals():
    x, gamma = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    q = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):       # not on the GPU
        te.te_rmsnorm_fp8(x, gamma, EPS, te.E4M3, torch.ones(1), q)
    with pytest.raises(TypeError):        # dtype of x
        te.te_rmsnorm_fp8(x.half(), gamma, EPS, te.E4M3, torch.ones(1), q)
    with pytest.raises(ValueError):       # a transposed view
        te.te_rmsnorm_fp8(torch.zeros(64, 4, dtype=torch.bfloat16).t(), gamma, EPS, te.E4M3, torch.ones(1), q)
    with pytest.raises(ValueError):       # three dimensions
        te.te_rmsnorm_mxfp8(x[None], gamma, EPS, q, q)
    with pytest.raises(ValueError):
        te.te_rmsnorm_bwd(x, x[0], gamma, torch.ones(4), x, gamma, torch.ones(4 * 64))


def test_library_refusals():
    import ctypes
    L = te.lib()
    ok, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)     # never dereferenced

    def fp8(x=ok, dt=te.BF16, rows=4, cols=64, res=None, gamma=ok, eps=1e-5, fmt=te.E4M3, scale=ok, q=ok, y=None):
        return L.te_rmsnorm_fp8(x, dt, rows, cols, res, gamma, eps, fmt, scale, q, y, None, None, None, None, None)

    assert fp8(cols=24) == 2 and fp8(cols=0) == 2 and fp8(cols=16400) == 2 and fp8(rows=-1) == 2
    assert fp8(dt=te.E4M3) == 4 and fp8(fmt=te.E2M1) == 4
    assert fp8(eps=-1.0) == 8 and fp8(eps=float("nan")) == 8 and fp8(eps=float("inf")) == 8
    assert fp8(gamma=None) == 1 and fp8(scale=None) == 1 and fp8(x=None) == 1
    assert fp8(x=odd) == 3 and fp8(res=odd) == 3 and fp8(q=odd) == 3 and fp8(y=odd) == 3 and fp8(gamma=odd) == 3
    assert fp8(x=None, rows=0) == 0

    def mx(cols=64, q=ok, s=ok, rows=4):
        return L.te_rmsnorm_mxfp8(ok, te.BF16, rows, cols, None, ok, 1e-5, q, s, None, None, None, None)

    assert mx(cols=48) == 2 and mx(q=None) == 1 and mx(s=None) == 1 and mx(q=odd) == 3 and mx(s=odd) == 3
    assert mx(rows=0) == 0
    need = te.te_rmsnorm_bwd_workspace_bytes(4, 64)
    assert need == 4 * 64 * 4 and te.te_rmsnorm_bwd_workspace_bytes(10 ** 6, 64) == 512 * 64 * 4

    def bwd(dy=ok, s=ok, rows=4, cols=64, dgamma=ok, dx=ok, ws=ok, n=need, dres=None):
        return L.te_rmsnorm_bwd(dy, s, te.BF16, rows, cols, ok, ok, dres, dx, dgamma, ws, n, None)

    assert bwd(n=need - 1) == 2 and bwd(cols=40) == 2 and bwd(dy=None) == 1 and bwd(ws=None) == 1
    assert bwd(dgamma=None) == 1 and bwd(dx=odd) == 3 and bwd(dres=odd) == 3 and bwd(ws=odd) == 3
