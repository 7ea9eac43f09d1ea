"""LayerNorm with the residual's addition, its 8-bit outputs and its gradient, against the 64-bit oracle.

Tolerances count roundings.  E = 2^-24 is half a step of fp32, 2^-8 of bf16, 2^-4 of E4M3 and 2^-3 of E5M2
(relative).  With A the mean of a row's |s|: a sum over the row is built from at most 32 terms per lane pair, a
5-step butterfly and 16 warps' sums, so mu is within 64 E A; s is one rounding of x + residual, E |s|.  The sum of
squares about a mean that is d off is n d^2 off, and each square's root is E |s| + E |s - mu| off, so rsigma is
within 44 E + 2 E rms(s) rsigma + (64 E A rsigma)^2 relative, and y = ((s - mu) rsigma) gamma + beta adds four
roundings of the product and one of the sum before its own.
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle.layernorm import add_layernorm, layernorm_bwd
from tests import gpu_util as G
from tests.kernel_names import launched
from tests.test_gpu_gated import _codes

E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": E}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-5


def _np(t):
    return t.detach().cpu().double().numpy()


def _inputs(rows, cols, dtype, seed=0, residual=True, mean=0.5):
    g = torch.Generator().manual_seed(seed + 7 * rows + cols)
    x = torch.randn(rows, cols, generator=g)
    r = torch.randn(rows, cols, generator=g) * (1 + 30 * (torch.rand(cols, generator=g) < 0.02)) + mean
    gamma, beta = 1 + 0.2 * torch.randn(cols, generator=g), 0.3 * torch.randn(cols, generator=g)
    return (x.to(DT[dtype]).to(G.DEV), r.to(DT[dtype]).to(G.DEV) if residual else None, gamma.to(G.DEV), beta.to(G.DEV))


def _errors(s, y, gamma, mu, rs):
    """Absolute errors of mu, of rsigma (relative), and of y before its rounding."""
    dmu = 64 * E * np.abs(s).mean(1)
    rel = 44 * E + 2 * E * np.sqrt((s ** 2).mean(1)) * rs + (dmu * rs) ** 2
    c = np.abs(s - mu[:, None])
    dy = np.abs(gamma) * rs[:, None] * (E * np.abs(s) + dmu[:, None] + c * (rel[:, None] + 4 * E)) + E * np.abs(y)
    return dmu, rel, dy


def _forward(x, r, gamma, beta, fmt=None, scale=1.0, stream=None):
    """Every output of the FP8 (fmt) or MXFP8 (None) call, in poisoned buffers."""
    rows, cols = x.shape
    o = dict(q=G.u8(rows, cols), y=torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=G.DEV),
             res_out=torch.full_like(x, 7.0), mu=torch.full((rows,), -1.0, device=G.DEV),
             rsigma=torch.full((rows,), -1.0, device=G.DEV))
    common = dict(residual=r, res_out=o["res_out"], y=o["y"], mu=o["mu"], rsigma=o["rsigma"], stream=stream)
    if fmt:
        o["amax"], o["inv"], sc = G.scalar(-1.0), G.scalar(-1.0), G.scalar(float(scale))
        o["call"] = lambda st=None: te.te_add_layernorm_fp8(
            x, gamma, beta, EPS, te.E4M3 if fmt == "e4m3" else te.E5M2, sc, o["q"], amax_out=o["amax"],
            scale_inv_out=o["inv"], **{**common, "stream": st or stream})
    else:
        o["s"] = G.u8(te.te_scale_bytes(te.E8M0, rows, cols))
        o["call"] = lambda st=None: te.te_add_layernorm_mxfp8(x, gamma, beta, EPS, o["q"], o["s"],
                                                              **{**common, "stream": st or stream})
    o["call"]()
    torch.cuda.synchronize()
    G.check_no_device_error()
    return o


def _check(x, r, gamma, beta, dtype, fmt):
    s64, y64, mu64, rs64 = add_layernorm(_np(x), _np(gamma), _np(beta), EPS, None if r is None else _np(r))
    scale = np.float32(FMAX[fmt] / (0.7 * np.abs(y64).max())) if fmt else None       # some values saturate
    o = _forward(x, r, gamma, beta, fmt, scale)
    dmu, rel, dy = _errors(s64, y64, _np(gamma), mu64, rs64)
    assert np.all(np.abs(_np(o["res_out"]) - s64) <= (HALF[dtype] + E) * np.abs(s64))
    assert np.all(np.abs(_np(o["mu"]) - mu64) <= dmu)
    assert np.all(np.abs(_np(o["rsigma"]) - rs64) <= rel * rs64)
    assert np.all(np.abs(_np(o["y"]) - y64) <= 2.0 ** -8 * (np.abs(y64) + dy) + dy)
    if fmt:
        sc = float(scale)
        _codes(o["q"].cpu().numpy(), y64 * sc, dy * sc + E * np.abs(y64) * sc, fmt, "q")
        assert abs(o["amax"].item() - np.abs(y64).max()) <= dy.max()
        assert np.float32(o["inv"].item()) == np.float32(1.0) / scale
    else:
        rows, cols = x.shape
        raw = o["s"].cpu().numpy()
        s = te.te_scale_unswizzle(te.E8M0, rows, cols, raw).astype(np.int64)
        top, slack = (a.reshape(rows, cols // 32, 32) for a in (np.abs(y64), dy))
        lo = np.floor(np.log2((top - slack).max(-1).clip(1e-30))) + 119
        hi = np.floor(np.log2((top + slack).max(-1))) + 119
        assert np.all((s >= lo) & (s <= hi))
        assert int(raw.astype(np.int64).sum()) == int(s.sum())               # padding is zero
        mul = np.exp2(127.0 - np.repeat(s, 32, 1))
        _codes(o["q"].cpu().numpy(), y64 * mul, dy * mul, "e4m3", "q")
    return o


# one to sixteen warps a row, whole and ragged, and (the last six) several rows a group with an unequal last pass
SHAPES = [(1, 16), (1, 4096), (3, 48), (17, 1024), (9, 1040), (33, 2048), (5, 2064), (7, 5120), (3, 8208), (2, 16384),
          (5003, 512), (5003, 1024), (2600, 1040), (1501, 4096), (701, 8192), (331, 16384)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,residual,fmt", [("bf16", True, "e4m3"), ("fp32", True, "e5m2"), ("bf16", False, "e5m2")])
def test_fp8(rows, cols, dtype, residual, fmt):
    x, r, gamma, beta = _inputs(rows, cols, dtype, residual=residual)
    _check(x, r, gamma, beta, dtype, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (127, 160), (129, 1024), (40, 1056), (5, 8224),
                                       (2, 16384), (5003, 512), (2600, 1056), (1501, 4096), (331, 16384)])
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp32", False)])
def test_mxfp8(rows, cols, dtype, residual):
    x, r, gamma, beta = _inputs(rows, cols, dtype, 1, residual)
    _check(x, r, gamma, beta, dtype, None)


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [768, 4096, 16384])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_mean_far_from_zero(cols, dtype):
    """A mean of a hundred deviations: sums of squares about zero would have lost the variance."""
    x, r, gamma, beta = _inputs(40, cols, dtype, 2, mean=100.0)
    _check(x, r, gamma, beta, dtype, "e4m3")


@pytest.mark.gpu
def test_rows_walk():
    """More rows than row groups, in a captured launch of the same call."""
    x, r, gamma, beta = _inputs(1501, 4096, "bf16")
    o = _forward(x, r, gamma, beta, "e4m3")
    (ctas,) = [n for name, n in launched(lambda st: o["call"](st)) if "layernorm_rows_kernel" in name]
    assert 2 * ctas < 1501


@pytest.mark.gpu
def test_optional_outputs_and_in_place():
    x, r, gamma, beta = _inputs(40, 1024, "bf16", 2)
    want = _forward(x, r, gamma, beta, "e4m3", 3.0)
    y = torch.empty_like(x)
    te.te_add_layernorm_fp8(x, gamma, beta, EPS, te.E4M3, residual=r, y=y)      # bf16 only: no scale needed
    torch.cuda.synchronize()
    assert torch.equal(y, want["y"])
    for target in ("x", "r"):
        a, b, q = x.clone(), r.clone(), G.u8(40, 1024)
        te.te_add_layernorm_fp8(a, gamma, beta, EPS, te.E4M3, G.scalar(3.0), q, residual=b,
                                res_out=a if target == "x" else b)
        torch.cuda.synchronize()
        assert torch.equal(a if target == "x" else b, want["res_out"]) and torch.equal(q, want["q"])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", None])
def test_special_values(fmt):
    """A row of one value gives beta, infinities and NaN stay in their rows; the amax does not lose a NaN."""
    x, _, gamma, beta = _inputs(6, 256, "fp32", 3)
    x[1] = 4.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] *= 1e-30
    o = _forward(x, None, gamma, beta, fmt)
    yn = o["y"].float().cpu().numpy()
    s64, y64, mu64, rs64 = add_layernorm(_np(x)[[0, 1, 4, 5]], _np(gamma), _np(beta), EPS)
    _, _, dy = _errors(s64, y64, _np(gamma), mu64, rs64)
    assert np.all(np.abs(yn[[0, 1, 4, 5]] - y64) <= 2.0 ** -8 * (np.abs(y64) + dy) + dy)
    assert torch.equal(o["y"][1], beta.bfloat16()) and np.isnan(yn[2]).all() and np.isnan(yn[3]).all()
    if fmt:
        assert np.isnan(o["amax"].item())


@pytest.mark.gpu
def test_no_rows():
    x, gamma = torch.empty(0, 64, dtype=torch.bfloat16, device=G.DEV), torch.ones(64, device=G.DEV)
    amax, inv, none = G.scalar(-1.0), G.scalar(-1.0), torch.empty(0, device=G.DEV)
    q = torch.empty(0, 64, dtype=torch.uint8, device=G.DEV)
    te.te_add_layernorm_fp8(x, gamma, gamma, EPS, te.E4M3, G.scalar(4.0), q, amax_out=amax, scale_inv_out=inv)
    te.te_add_layernorm_mxfp8(x, gamma, gamma, EPS, q, q.view(-1))
    dgamma, dbeta = torch.full((64,), 3.0, device=G.DEV), torch.full((64,), 3.0, device=G.DEV)
    te.te_layernorm_bwd(x, x, gamma, none, none, x.clone(), dgamma, dbeta, none)
    torch.cuda.synchronize()
    assert amax.item() == 0 and inv.item() == 0.25 and not dgamma.any() and not dbeta.any()


def _bwd_inputs(rows, cols, dtype, residual, seed=4):
    x, _, gamma, _ = _inputs(rows, cols, dtype, seed)
    g = torch.Generator().manual_seed(seed)
    dy = (torch.randn(rows, cols, generator=g) * 1e-3).bfloat16().to(G.DEV)
    dres = (torch.randn(rows, cols, generator=g) * 1e-3).to(DT[dtype]).to(G.DEV) if residual else None
    mu = x.double().mean(1)
    rs = torch.rsqrt((x.double() - mu[:, None]).square().mean(1) + EPS).float()
    return dy, x, gamma, mu.float(), rs, dres


def _backward(dy, x, gamma, mu, rs, dres, dx=None, stream=None):
    rows, cols = x.shape
    dx = torch.full_like(x, 7.0) if dx is None else dx
    dgamma, dbeta = (torch.full((cols,), 7.0, device=G.DEV) for _ in range(2))
    ws = torch.full((te.te_layernorm_bwd_workspace_bytes(rows, cols) // 4,), float("nan"), device=G.DEV)
    te.te_layernorm_bwd(dy, x, gamma, mu, rs, dx, dgamma, dbeta, ws, dres=dres, stream=stream)
    torch.cuda.synchronize()
    G.check_no_device_error()
    return dx, dgamma, dbeta


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 4096), (700, 2048), (331, 8208)])
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("fp32", True), ("bf16", False), ("fp32", False)])
def test_backward(rows, cols, dtype, residual):
    dy, x, gamma, mu, rs, dres = _bwd_inputs(rows, cols, dtype, residual)
    dx, dgamma, dbeta = _backward(dy, x, gamma, mu, rs, dres)
    ds64, dg64, db64 = layernorm_bwd(_np(dy), _np(x), _np(gamma), _np(mu), _np(rs), None if dres is None else _np(dres))
    # per element: xhat (2 roundings), p and the means (64 E of their absolute terms), three fused steps
    xhat = np.abs(_np(x) - _np(mu)[:, None]) * _np(rs)[:, None]
    p = np.abs(_np(dy) * _np(gamma))
    size = _np(rs)[:, None] * (p + p.mean(1, keepdims=True) + xhat * (p * xhat).mean(1, keepdims=True))
    tol = 72 * E * size + (HALF[dtype] + E) * (np.abs(ds64) + 72 * E * size)
    assert np.all(np.abs(_np(dx) - ds64) <= tol), float(np.max(np.abs(_np(dx) - ds64) / tol))
    assert np.all(np.abs(_np(dgamma) - dg64) <= (rows + 5) * E * (np.abs(_np(dy)) * xhat).sum(0))
    assert np.all(np.abs(_np(dbeta) - db64) <= rows * E * np.abs(_np(dy)).sum(0))


@pytest.mark.gpu
def test_backward_in_place_streams_graphs_and_repeats():
    dy, x, gamma, mu, rs, dres = _bwd_inputs(2000, 768, "bf16", True)
    want = _backward(dy, x, gamma, mu, rs, dres)
    a = dres.clone()
    b = x.clone()
    for got in (_backward(dy, x, gamma, mu, rs, a, dx=a), _backward(dy, b, gamma, mu, rs, dres, dx=b),
                _backward(dy, x, gamma, mu, rs, dres, stream=torch.cuda.Stream())):
        assert all(torch.equal(m, n) for m, n in zip(got, want))
    ws = torch.empty(te.te_layernorm_bwd_workspace_bytes(2000, 768) // 4, device=G.DEV)
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):      # the sums start while the rows' kernel drains, and the next call behind them
            te.te_layernorm_bwd(dy, x, gamma, mu, rs, *out, ws, dres=dres)
        copies = [t.clone() for t in out]
    for _ in range(3):
        for t in out:
            t.zero_()
        ws.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(copies, want))


# ---- refusals: nothing reaches the GPU --------------------------------------------------------

def test_wrapper_refusals():
    x, g = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    q = torch.zeros(4, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):       # not on the GPU
        te.te_add_layernorm_fp8(x, g, g, EPS, te.E4M3, torch.ones(1), q)
    with pytest.raises(TypeError):        # dtype of x
        te.te_add_layernorm_fp8(x.half(), g, g, EPS, te.E4M3, torch.ones(1), q)
    with pytest.raises(ValueError):       # a transposed view
        te.te_add_layernorm_fp8(torch.zeros(64, 4, dtype=torch.bfloat16).t(), g, g, EPS, te.E4M3, torch.ones(1), q)
    with pytest.raises(ValueError):       # three dimensions
        te.te_add_layernorm_mxfp8(x[None], g, g, EPS, q, q)
    with pytest.raises(ValueError):
        te.te_layernorm_bwd(x, x[0], g, torch.ones(4), torch.ones(4), x, g, g, torch.ones(8 * 64))


def test_library_refusals():
    import ctypes
    L = te.lib()
    ok, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)     # never dereferenced

    def fp8(x=ok, dt=te.BF16, rows=4, cols=64, res=None, g=ok, b=ok, eps=1e-5, fmt=te.E4M3, scale=ok, q=ok, y=None):
        return L.te_add_layernorm_fp8(x, dt, rows, cols, res, g, b, eps, fmt, scale, q, y, None, None, None, None, None, None)

    assert fp8(cols=24) == 2 and fp8(cols=0) == 2 and fp8(cols=16400) == 2 and fp8(rows=-1) == 2
    assert fp8(dt=te.E4M3) == 4 and fp8(fmt=te.E2M1) == 4
    assert fp8(eps=-1.0) == 8 and fp8(eps=float("nan")) == 8 and fp8(eps=float("inf")) == 8
    assert fp8(g=None) == 1 and fp8(b=None) == 1 and fp8(scale=None) == 1 and fp8(x=None) == 1
    for name in ("x", "res", "q", "y", "g", "b"):
        assert fp8(**{name: odd}) == 3
    assert fp8(x=None, rows=0) == 0

    def mx(cols=64, q=ok, s=ok, rows=4):
        return L.te_add_layernorm_mxfp8(ok, te.BF16, rows, cols, None, ok, ok, 1e-5, q, s, None, None, None, None, None)

    assert mx(cols=48) == 2 and mx(q=None) == 1 and mx(s=None) == 1 and mx(q=odd) == 3 and mx(s=odd) == 3
    assert mx(rows=0) == 0
    need = te.te_layernorm_bwd_workspace_bytes(4, 64)
    assert need == 8 * 64 * 4 and te.te_layernorm_bwd_workspace_bytes(10 ** 6, 64) == 1024 * 64 * 4

    def bwd(dy=ok, s=ok, rows=4, cols=64, dg=ok, db=ok, dx=ok, ws=ok, n=need, dres=None, mu=ok):
        return L.te_layernorm_bwd(dy, s, te.BF16, rows, cols, ok, mu, ok, dres, dx, dg, db, ws, n, None)

    assert bwd(n=need - 1) == 2 and bwd(cols=40) == 2 and bwd(dy=None) == 1 and bwd(ws=None) == 1 and bwd(mu=None) == 1
    assert bwd(dg=None) == 1 and bwd(db=None) == 1 and bwd(dx=odd) == 3 and bwd(dres=odd) == 3 and bwd(ws=odd) == 3
