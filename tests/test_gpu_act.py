"""The linear with bias, activation and residual (every operand kind, activation and output) and its backward
passes, against the 64-bit oracle on the operands' own values.

Tolerances.  A product over K terms is within (K + 4) 2^-23 S of the exact one, S the sum of the terms' sizes
(fp32 accumulation, whatever its order, and alpha); the bias's addition rounds once; the activations' slopes are
below 1.2 and their sigmoid within (8 + 4 |z|) 2^-23 (see test_gpu_gated); the residual's addition rounds once; an
output of half a step r (bf16 2^-8, E4M3 2^-4, E5M2 2^-3, fp32 2^-24) adds r of the value.
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle.act import act_dgrad, act_grad, linear_act
from tests import gpu_util as G
from tests.test_gpu_gated import BF, E23, FMAX, FMT, Operand, Out, _codes

ACT = {"none": te.ACT_NONE, "relu": te.ACT_RELU, "silu": te.ACT_SILU, "gelu": te.ACT_GELU}
YT = {"y": torch.bfloat16, "y32": torch.float32}


def _inputs(T, K, N, seed):
    rng = np.random.default_rng(seed + T + 3 * K + 7 * N)
    return rng.standard_normal((T, K)), rng.standard_normal((N, K)) * (1.5 / np.sqrt(K))


def _sigmoid_error(z, actk):
    if actk in ("none", "relu"):
        return np.zeros_like(z)
    return (8 + 4 * (np.abs(z) if actk == "silu" else 2 * np.abs(z) * (1 + 0.05 * z * z))) * E23


def forward(kind, T, K, N, actk, outs, seed=0, fmt="e4m3", stream=None, ops=None):
    """Outputs of one call.  outs: of "z", "y" or "y32", "q", "bias", "res"."""
    a, b = _inputs(T, K, N, seed)
    x, w = ops or (Operand(a, kind), Operand(b, kind))
    rng = np.random.default_rng(seed + T * N)
    bias = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(G.DEV) if "bias" in outs else None
    yt = YT["y32" if "y32" in outs else "y"]
    res = torch.from_numpy(rng.standard_normal((T, N)) * 2).to(yt).to(G.DEV) if "res" in outs else None
    o = dict(x=x, w=w, bias=bias, res=res, z=Out(T, N) if "z" in outs else None,
             y=Out(T, N, dtype=yt) if "y" in outs or "y32" in outs else None)
    more = dict(bias=bias, residual=res, z=o["z"] and o["z"].t, y=o["y"] and o["y"].t)
    if "q" in outs:
        o["q"] = Out(T, N, dtype=torch.uint8)
        more["q"] = o["q"].t
        if kind == "fp8":
            o["amax"], o["inv"], o["scale"] = G.scalar(-1.0), G.scalar(-1.0), np.float32(FMAX[fmt] / 3.0)   # some saturate
            more.update(q_fmt=FMT[fmt], q_scale=G.scalar(float(o["scale"])), q_amax=o["amax"], q_scale_inv=o["inv"])
        else:
            o["s"] = Out(te.te_scale_bytes(te.E8M0, T, N), dtype=torch.uint8)
            more["s_q"] = o["s"].t

    def call(st=None):
        A, kw = ACT[actk], {**more, "stream": st or stream}
        if kind == "bf16":
            te.te_act_gemm_bf16(x.q, w.q, A, **kw)
        elif kind == "fp8":
            te.te_act_gemm_fp8(x.q, FMT[x.fmt], w.q, FMT[w.fmt], x.inv, w.inv, A, **kw)
        elif kind == "mxfp8":
            te.te_act_gemm_mxfp8(x.q, x.s, w.q, w.s, A, **kw)
        else:
            te.te_act_gemm_nvfp4(x.q, x.s, x.g, w.q, w.s, w.g, A, **kw)

    o["call"] = call
    call()
    torch.cuda.synchronize()
    G.check_no_device_error()
    return o


def check_forward(kind, T, K, N, actk, outs, fmt="e4m3", ops=None, seed=0):
    o = forward(kind, T, K, N, actk, outs, fmt=fmt, ops=ops, seed=seed)
    num = lambda t: None if t is None else t.cpu().double().numpy()   # noqa: E731
    y64, z64, a64 = linear_act(o["x"].v, o["w"].v, actk, num(o["bias"]), num(o["res"]))
    S = np.abs(o["x"].v) @ np.abs(o["w"].v).T
    dz = (K + 4) * E23 * S + E23 * np.abs(z64)
    da = 1.2 * dz + _sigmoid_error(z64, actk) * np.abs(a64)
    if o["z"]:
        assert np.all(np.abs(o["z"].np() - z64) <= BF * (np.abs(z64) + dz) + dz), "z"
    if o["y"]:
        err = da + (E23 * np.abs(y64) if o["res"] is not None else 0.0)
        half = BF if o["y"].t.dtype == torch.bfloat16 else E23 / 2
        assert np.all(np.abs(o["y"].np() - y64) <= half * (np.abs(y64) + err) + err), "y"
    if "q" in o and kind == "fp8":
        sc = float(o["scale"])
        _codes(o["q"].np(), a64 * sc, da * sc + np.abs(a64) * sc * E23, fmt, "q")
        assert abs(o["amax"].item() - np.abs(a64).max()) <= da.max()
        assert np.float32(o["inv"].item()) == np.float32(1) / o["scale"]
    elif "q" in o:
        raw = o["s"].np()
        s = te.te_scale_unswizzle(te.E8M0, T, N, raw).astype(np.int64)
        top, slack = (v.reshape(T, -1, 32) for v in (np.abs(a64), da))
        with np.errstate(divide="ignore"):
            lo = np.maximum(np.floor(np.log2((top - slack).max(-1).clip(0))) + 119, 0)
            hi = np.maximum(np.floor(np.log2((top + slack).max(-1))) + 119, 0)
        assert np.all((s >= lo) & (s <= hi)), "scales"
        assert int(raw.astype(np.int64).sum()) == int(s.sum()), "padding"
        mul = np.exp2(127.0 - np.repeat(s, 32, 1))
        _codes(o["q"].np(), a64 * mul, da * mul, "e4m3", "q")
    return o


def same_again(o):
    """A second call on the same operands writes the same bits."""
    names = [n for n in ("z", "y", "q", "s", "amax") if o.get(n) is not None]
    get = lambda n: o[n].t if isinstance(o[n], Out) else o[n]   # noqa: E731
    first = [get(n).clone() for n in names]
    for n in names:
        get(n).zero_()
    o["call"]()
    torch.cuda.synchronize()
    for n, f in zip(names, first):
        assert torch.equal(get(n), f), n


# one token to several tiles of tokens; widths that end inside a box, a tile, a k-step
GENERAL = [(1, 16, 16), (1, 208, 272), (2, 80, 48), (15, 64, 112), (17, 400, 144), (33, 768, 256), (127, 48, 128),
           (129, 320, 400), (256, 64, 144), (257, 96, 1040), (385, 128, 64)]
BLOCK = [(1, 32, 32), (3, 96, 160), (31, 416, 128), (64, 256, 416), (129, 160, 96), (300, 544, 672)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", GENERAL)
@pytest.mark.parametrize("actk,outs", [("gelu", ("y", "bias")), ("silu", ("z", "y", "bias")), ("none", ("y", "bias", "res")),
                                       ("relu", ("z", "y", "res")), ("none", ("y32", "bias", "res")),
                                       ("gelu", ("z", "y32", "bias", "res")), ("relu", ("z", "y32")), ("silu", ("z",))])
def test_bf16(T, K, N, actk, outs):
    check_forward("bf16", T, K, N, actk, outs)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", GENERAL)
@pytest.mark.parametrize("actk,outs,fmt", [("gelu", ("q", "bias"), "e4m3"), ("relu", ("z", "y", "q", "bias"), "e5m2"),
                                           ("silu", ("z", "y32", "q"), "e4m3"), ("none", ("y", "bias", "res"), "e4m3"),
                                           ("none", ("y32", "res"), "e4m3")])
def test_fp8(T, K, N, actk, outs, fmt):
    check_forward("fp8", T, K, N, actk, outs, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", BLOCK)
@pytest.mark.parametrize("kind,actk,outs", [("mxfp8", "gelu", ("q", "bias")), ("mxfp8", "relu", ("z", "y", "q", "bias")),
                                            ("mxfp8", "none", ("y", "bias", "res")), ("mxfp8", "silu", ("z", "y32", "q")),
                                            ("nvfp4", "gelu", ("z", "y", "bias")), ("nvfp4", "none", ("y32", "bias", "res")),
                                            ("nvfp4", "silu", ("z", "y", "res"))])
def test_block_scaled(T, K, N, kind, actk, outs):
    check_forward(kind, T, K, N, actk, outs)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,K,N", [(1, 32, 16), (5, 96, 48), (70, 160, 144), (300, 96, 400)])
def test_block_scaled_columns_of_sixteen(kind, T, K, N):
    """Without an 8-bit output N is any multiple of 16."""
    check_forward(kind, T, K, N, "gelu", ("z", "y", "bias"))
    check_forward(kind, T, K, N, "none", ("y32", "bias", "res"))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,outs", [("bf16", ("z", "y", "res", "bias")), ("bf16", ("y32", "res")), ("fp8", ("z", "y", "q", "bias")),
                                       ("mxfp8", ("z", "y", "q", "bias")), ("mxfp8", ("y", "res")), ("nvfp4", ("z", "y32", "bias", "res"))])
def test_several_tiles_per_cta(kind, outs):
    """More tiles than CTA pairs: the rings, the accumulators and the staging boxes are used again."""
    check_forward(kind, 2100 if kind in ("bf16", "fp8") else 2080, 320, 3328, "gelu", outs)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 4096, 4960), (8, 2064, 160), (9, 1040, 2464), (16, 4112, 64), (24, 4096, 96),
                                   (32, 2096, 2496), (25, 4096, 64), (20, 4096, 160), (40, 128, 20000), (64, 2064, 544),
                                   (31, 6000, 16), (3, 16400, 64), (1, 16400, 2432), (5, 96, 20000), (128, 4112, 272)])
@pytest.mark.parametrize("kind,actk,outs,fmt", [("bf16", "gelu", ("z", "y", "bias"), "e4m3"),
                                                ("bf16", "none", ("y32", "bias", "res"), "e4m3"),
                                                ("fp8", "relu", ("z", "y", "q"), "e4m3"), ("fp8", "gelu", ("q", "bias"), "e5m2"),
                                                ("fp8", "silu", ("y", "res"), "e4m3")])
def test_few_tokens(T, K, N, kind, actk, outs, fmt):
    """Long rows and more units of columns than SMs, and few columns on a long row."""
    same_again(check_forward(kind, T, K, N, actk, outs, fmt))


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 4128, 2560), (8, 8256, 256), (5, 160, 9984), (2, 64, 5120), (9, 4128, 288),
                                   (7, 13696, 224), (30, 4128, 4096), (64, 2048, 20000), (61, 800, 9728), (90, 4128, 608),
                                   (128, 8224, 256)])
@pytest.mark.parametrize("kind,actk,outs", [("mxfp8", "gelu", ("q", "bias")), ("mxfp8", "relu", ("z", "y", "q", "bias")),
                                            ("mxfp8", "none", ("y32", "bias", "res")), ("nvfp4", "silu", ("z", "y", "bias")),
                                            ("nvfp4", "none", ("y", "res"))])
def test_few_tokens_block_scaled(T, K, N, kind, actk, outs):
    same_again(check_forward(kind, T, K, N, actk, outs))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 40, 200])
@pytest.mark.parametrize("fx,fw", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_fp8_operand_formats(T, fx, fw):
    a, b = _inputs(T, 208, 144, 5)
    check_forward("fp8", T, 208, 144, "silu", ("y", "bias"), ops=(Operand(a, "fp8", fx), Operand(b, "fp8", fw)))


# contractions long enough for a tile to be shared by two or four CTA pairs, with few tiles (four), more (two), ragged
# edges and parts of unequal length, and a last, partial wave behind full ones
@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(140, 3216, 32), (150, 3200, 288), (129, 4112, 544), (300, 6160, 3200), (513, 3216, 800),
                                   (165, 8208, 256), (2100, 3216, 2560), (1300, 6160, 4096)])
@pytest.mark.parametrize("kind,actk,outs,fmt", [("bf16", "silu", ("z", "y", "res"), "e4m3"), ("bf16", "none", ("y32", "res", "bias"), "e4m3"),
                                                ("fp8", "gelu", ("z", "y", "q", "bias"), "e4m3"), ("fp8", "relu", ("q",), "e5m2")])
def test_shared_contraction(T, K, N, kind, actk, outs, fmt):
    same_again(check_forward(kind, T, K, N, actk, outs, fmt))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 100, 300])
@pytest.mark.parametrize("kind,yt", [("bf16", "y"), ("fp8", "y32"), ("mxfp8", "y32"), ("nvfp4", "y")])
def test_residual_in_place(T, kind, yt):
    """y over the residual."""
    o = forward(kind, T, 224, 416, "gelu", (yt, "bias", "res"))
    same = o["res"].clone()
    x, w, kw = o["x"], o["w"], dict(bias=o["bias"], residual=same, y=same)
    if kind == "bf16":
        te.te_act_gemm_bf16(x.q, w.q, te.ACT_GELU, **kw)
    elif kind == "fp8":
        te.te_act_gemm_fp8(x.q, te.E4M3, w.q, te.E4M3, x.inv, w.inv, te.ACT_GELU, **kw)
    elif kind == "mxfp8":
        te.te_act_gemm_mxfp8(x.q, x.s, w.q, w.s, te.ACT_GELU, **kw)
    else:
        te.te_act_gemm_nvfp4(x.q, x.s, x.g, w.q, w.s, w.g, te.ACT_GELU, **kw)
    torch.cuda.synchronize()
    assert torch.equal(same, o["y"].t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(1, 64), (20, 64), (100, 4096), (300, 64)])
@pytest.mark.parametrize("actk", ["relu", "gelu"])
def test_special_values_stay_in_their_row(T, K, actk):
    a, b = _inputs(T, K, 160, 1)
    a[T // 2, 3] = np.nan
    o = forward("bf16", T, K, 160, actk, ("z", "y"), ops=(Operand(a, "bf16"), Operand(b, "bf16")))
    for n in ("z", "y"):
        v = o[n].np()
        assert np.isnan(v[T // 2]).all() and np.isfinite(np.delete(v, T // 2, 0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 20, 40, 100, 200])
@pytest.mark.parametrize("K", [64, 4096])
def test_what_is_not_finite_stays_out_of_the_rest(T, K):
    """A weight that is not finite makes the rows past the last token NaN inside a tile (zero times infinity), a
    token that is not makes the columns past the last one so: neither reaches the amax or the scales' padding."""
    a, b = _inputs(T, K, 144, 4)
    x, w = Operand(np.abs(a) + 0.1, "fp8"), Operand(b, "fp8", "e5m2")
    w.q[5, 7] = 0x7C                                           # +inf: z[:, 5] = +inf
    y, q, amax = Out(T, 144), Out(T, 144, dtype=torch.uint8), G.scalar(-1.0)

    def call():
        te.te_act_gemm_fp8(x.q, FMT[x.fmt], w.q, FMT[w.fmt], x.inv, w.inv, te.ACT_RELU, y=y.t, q=q.t, q_scale=G.scalar(1.0),
                           q_amax=amax)
        torch.cuda.synchronize()

    call()
    assert np.isposinf(y.np()[:, 5]).all() and np.isfinite(np.delete(y.np(), 5, 1)).all() and np.isposinf(amax.item())
    x, w = Operand(a, "fp8", "e5m2"), Operand(np.abs(b) + 0.01, "fp8")
    w.q.clamp_(min=1)                                          # no zero times infinity in the columns that are there
    x.q[T - 1, 3] = 0x7C
    call()
    assert np.isposinf(y.np()[T - 1]).all() and np.isposinf(amax.item())
    x, w = Operand(a, "mxfp8"), Operand(_inputs(T, K, 160, 4)[1], "mxfp8")
    w.q[5, 7] = 0x7F                                           # NaN
    q, s = Out(T, 160, dtype=torch.uint8), Out(te.te_scale_bytes(te.E8M0, T, 160), dtype=torch.uint8)
    te.te_act_gemm_mxfp8(x.q, x.s, w.q, w.s, te.ACT_SILU, q=q.t, s_q=s.t)
    torch.cuda.synchronize()
    raw = s.np()
    assert int(raw.astype(np.int64).sum()) == int(te.te_scale_unswizzle(te.E8M0, T, 160, raw).astype(np.int64).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 300])
def test_mxfp8_blocks_of_zeros(T):
    """ReLU leaves whole blocks zero: their scale is the smallest and their codes are zero."""
    a, b = _inputs(T, 64, 256, 6)
    x, w = Operand(np.abs(a), "mxfp8"), Operand(np.where(np.arange(256)[:, None] // 32 % 2, -np.abs(b), np.abs(b)), "mxfp8")
    o = check_forward("mxfp8", T, 64, 256, "relu", ("q", "y"), ops=(x, w))
    s = te.te_scale_unswizzle(te.E8M0, T, 256, o["s"].np())
    assert not s[:, 1::2].any() and s[:, 0::2].all() and not o["q"].np().reshape(T, 8, 32)[:, 1::2].any()


@pytest.mark.gpu
def test_no_tokens():
    w = torch.zeros(64, 32, dtype=torch.bfloat16, device=G.DEV)
    x = torch.zeros(0, 32, dtype=torch.bfloat16, device=G.DEV)
    te.te_act_gemm_bf16(x, w, te.ACT_GELU, y=torch.zeros(0, 64, dtype=torch.bfloat16, device=G.DEV))
    amax, inv, one = G.scalar(-1.0), G.scalar(-1.0), G.scalar(1.0)
    te.te_act_gemm_fp8(x.to(torch.uint8), te.E4M3, w.to(torch.uint8), te.E4M3, one, one, te.ACT_GELU,
                       q=torch.zeros(0, 64, dtype=torch.uint8, device=G.DEV), q_scale=G.scalar(4.0), q_amax=amax, q_scale_inv=inv)
    z, dy, w2 = (torch.zeros(*s, dtype=torch.bfloat16, device=G.DEV) for s in ((0, 64), (0, 16), (16, 64)))
    dw, db = torch.ones(64, 32, device=G.DEV), torch.ones(64, device=G.DEV)
    te.te_act_bwd_bf16(x, w, w2, dy, z, te.ACT_GELU, z.clone(), dbias=db, dx=x.clone(), dw=dw, accumulate=1)
    torch.cuda.synchronize()
    assert amax.item() == 0 and inv.item() == 0.25 and bool((dw == 1).all()) and not db.any()
    db.fill_(1.0)
    te.te_act_bwd_bf16(x, w, w2, dy, z, te.ACT_GELU, z.clone(), dw=dw)
    te.te_act_dgrad_fp8(dy.to(torch.uint8), te.E5M2, w2.t().contiguous().to(torch.uint8), te.E4M3, one, one, z, te.ACT_GELU,
                        z.clone(), dbias=db)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


# ---- backward -----------------------------------------------------------------------------------

def _dz_errors(dy_v, w2_v, z, actk, N):
    """Error of dz before its rounding."""
    ddh = np.abs(dy_v) @ np.abs(w2_v) * ((N + 4) * E23)
    if actk in ("none", "relu"):
        return ddh * np.abs(act_grad(z, actk))
    f = (4 * E23 + _sigmoid_error(z, actk))
    slope = np.abs(act_grad(z, actk)) + f * (1 + np.abs(z) * (1 if actk == "silu" else 1.6 * (1 + 0.14 * z * z)))
    dh = np.abs(dy_v @ w2_v) + ddh
    return ddh * slope + dh * (slope - np.abs(act_grad(z, actk)) + 4 * E23 * slope)


def check_dz(dz, db, dy_v, w2_v, z, actk, N):
    T = dz.shape[0]
    dz64, db64 = act_dgrad(dy_v, w2_v, z, actk)
    err = _dz_errors(dy_v, w2_v, z, actk, N) + 1e-38
    tol = BF * (np.abs(dz64) + err) + err
    assert np.all(np.abs(dz - dz64) <= tol), float(np.max(np.abs(dz - dz64) / tol))
    if db is not None:
        tol = err.sum(0) + (T + 4) * E23 * (np.abs(dz64) + err).sum(0)
        assert np.all(np.abs(db - db64) <= tol), float(np.max(np.abs(db - db64) / tol))


def _bwd_inputs(T, Fc, N, seed=0):
    rng = np.random.default_rng(seed + T + 5 * Fc + 11 * N)
    z = torch.from_numpy(rng.standard_normal((T, Fc)) * 1.5).bfloat16().to(G.DEV)
    return rng.standard_normal((T, N)) * 1e-3, rng.standard_normal((N, Fc)) * 0.05, z


def _workspace(T, Fc):
    return torch.full((te.te_act_dbias_workspace_bytes(T, Fc) // 4,), float("nan"), device=G.DEV)


def dgrad(kind, T, Fc, N, actk, ops=None, z=None, dz=None, dbias=True, stream=None):
    dy, w2, z_ = _bwd_inputs(T, Fc, N)
    z = z_ if z is None else z
    d, w = ops or (Operand(dy, kind, "e5m2"), Operand(w2.T, kind))
    o = Out(T, Fc) if dz is None else None
    db = torch.full((Fc,), 7.0, device=G.DEV) if dbias else None
    kw = dict(dbias=db, workspace=_workspace(T, Fc) if dbias else None, stream=stream)
    args = (None if actk == "none" else z, ACT[actk], o.t if o else dz)
    if kind == "fp8":
        te.te_act_dgrad_fp8(d.q, te.E5M2, w.q, te.E4M3, d.inv, w.inv, *args, **kw)
    elif kind == "mxfp8":
        te.te_act_dgrad_mxfp8(d.q, d.s, w.q, w.s, *args, **kw)
    else:
        te.te_act_dgrad_nvfp4(d.q, d.s, d.g, w.q, w.s, w.g, *args, **kw)
    if stream is None:
        torch.cuda.synchronize()
        G.check_no_device_error()
    return d, w, z, o, db


@pytest.mark.gpu
@pytest.mark.parametrize("T,Fc,N", [(1, 16, 32), (3, 272, 96), (33, 144, 64), (128, 48, 160), (130, 400, 64),
                                    (257, 1040, 32), (2100, 2640, 64)])
@pytest.mark.parametrize("kind,actk", [("fp8", "silu"), ("fp8", "none"), ("fp8", "gelu"), ("mxfp8", "gelu"), ("mxfp8", "relu"),
                                       ("nvfp4", "gelu"), ("nvfp4", "none")])
def test_dgrad(T, Fc, N, kind, actk):
    d, w, z, o, db = dgrad(kind, T, Fc, N, actk)
    check_dz(o.np(), db.cpu().double().numpy(), d.v, w.v.T, z.cpu().double().numpy(), actk, N)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp8", "mxfp8", "nvfp4"])
def test_dgrad_in_place_and_without_dbias(kind):
    _, _, z, o, db = dgrad(kind, 300, 400, 64, "silu")
    same = z.clone()
    dgrad(kind, 300, 400, 64, "silu", z=same, dz=same)
    assert torch.equal(same, o.t)
    _, _, _, p, none = dgrad(kind, 300, 400, 64, "silu", dbias=False)
    assert torch.equal(p.t, o.t) and none is None


@pytest.mark.gpu
@pytest.mark.parametrize("T,Fc,N", [(1, 16, 3216), (70, 272, 3200), (300, 144, 4112), (300, 2640, 6160)])
@pytest.mark.parametrize("actk", ["relu", "none"])
def test_shared_contraction_dgrad(T, Fc, N, actk):
    d, w, z, o, db = dgrad("fp8", T, Fc, N, actk)
    check_dz(o.np(), db.cpu().double().numpy(), d.v, w.v.T, z.cpu().double().numpy(), actk, N)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp8", "mxfp8"])
def test_a_weight_that_is_not_finite_reaches_its_own_column_only(kind):
    """The tile's rows past the last token are zero times it, and stay out of the sums."""
    dy, w2, z = _bwd_inputs(40, 160, 64)
    d, w = Operand(np.abs(dy), kind, "e5m2"), Operand(np.abs(w2).T, kind)
    d.q.clamp_(min=1)
    w.q[3, 9] = 0x7E                                           # the largest E4M3 code, times:
    if kind == "mxfp8":
        w.s[3 * 16 + 0] = 254                                  # 2^127: the products overflow
    else:
        w.inv.fill_(3e38)
        d.inv.fill_(3e38)
    zero = torch.ones_like(z)
    _, _, _, o, db = dgrad(kind, 40, 160, 64, "relu", ops=(d, w), z=zero)
    got = o.np()
    assert not np.isnan(got).any() and not bool(db.isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc,N", [(1, 16, 16, 16), (3, 208, 272, 80), (33, 64, 144, 48), (100, 768, 128, 768),
                                      (129, 80, 400, 64), (257, 96, 1040, 32), (1001, 48, 80, 112),
                                      (70, 96, 784, 1552), (1700, 304, 1600, 1600), (300, 400, 3200, 64),
                                      (2100, 2304, 2560, 1600)])
@pytest.mark.parametrize("actk,dwt", [("silu", torch.bfloat16), ("gelu", torch.float32), ("none", torch.bfloat16)])
def test_bwd_bf16(T, K, Fc, N, actk, dwt):
    dy, w2, z = _bwd_inputs(T, Fc, N)
    a, b = _inputs(T, K, Fc, 3)
    x, w, d, w2 = (Operand(v, "bf16") for v in (a, b, dy, w2))
    dz, dx, dw, db, ws = Out(T, Fc), Out(T, K), Out(Fc, K, dtype=dwt), torch.full((Fc,), 7.0, device=G.DEV), _workspace(T, Fc)
    z = None if actk == "none" else z
    te.te_act_bwd_bf16(x.q, w.q, w2.q, d.q, z, ACT[actk], dz.t, db, ws, dx.t, dw.t)
    torch.cuda.synchronize()
    got = dz.np()
    check_dz(got, db.cpu().double().numpy(), d.v, w2.v, np.zeros((T, Fc)) if z is None else z.cpu().double().numpy(), actk, N)
    # dx and dw from the dz that was written
    for out, want, size, n, half in ((dx, got @ w.v, np.abs(got) @ np.abs(w.v), Fc, BF),
                                     (dw, got.T @ x.v, np.abs(got).T @ np.abs(x.v), T, BF if dwt is torch.bfloat16 else E23)):
        tol = half * np.abs(want) + (n + 4) * E23 * (1 + half) * size + 1e-38
        assert np.all(np.abs(out.np() - want) <= tol)
    if dwt is torch.float32:
        first = dw.t.clone()
        te.te_act_bwd_bf16(x.q, w.q, w2.q, d.q, z, ACT[actk], dz.t, dw=dw.t, accumulate=1)
        torch.cuda.synchronize()
        assert torch.equal(dw.t, first + first)
    G.check_no_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc,N", [(1001, 768, 2048, 768), (60, 64, 1040, 2048), (3000, 1024, 1024, 256),
                                      (2100, 2304, 2560, 1600)])
def test_bwd_overlap_and_graph(T, K, Fc, N):
    """dX, dbias and dW overlap and start while dZ's kernel drains: twenty calls in a row, eager and in a graph, give
    the bits that calls on their own give, with every set of outputs, and what follows in the stream sees them all."""
    dy, w2, z = _bwd_inputs(T, Fc, N, 6)
    a, b = _inputs(T, K, Fc, 6)
    x, w, d, w2 = (torch.from_numpy(v).bfloat16().to(G.DEV) for v in (a, b, dy, w2))
    bufs = [(torch.empty(T, Fc, dtype=torch.bfloat16, device=G.DEV), torch.empty(Fc, device=G.DEV), torch.empty_like(x),
             torch.empty_like(w), _workspace(T, Fc)) for _ in range(2)]

    def call(scale, i, what=("db", "dx", "dw")):
        g, db, dx, dw, ws = bufs[i]
        te.te_act_bwd_bf16(x, w, w2, d * scale, z, te.ACT_SILU, g, db if "db" in what else None, ws if "db" in what else None,
                           dx if "dx" in what else None, dw if "dw" in what else None)
        return [t.clone() for t, n in ((g, ""), (db, "db"), (dx, "dx"), (dw, "dw")) if not n or n in what]

    for what in (("db", "dx", "dw"), ("db", "dw"), ("db", "dx"), ("db",), ("dx", "dw")):
        want = []
        for i in range(6):
            want.append(call(2.0 ** (i % 3), 0, what))
            torch.cuda.synchronize()
        got = [call(2.0 ** (i % 3), i % 2, what) for i in range(18)]
        torch.cuda.synchronize()
        for i, q in enumerate(got):
            assert all(torch.equal(m, n) for m, n in zip(want[i % 6], q)), (what, i)
    want = call(1.0, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, db, dx, dw, ws = bufs[1]
        for i in range(5):
            te.te_act_bwd_bf16(x, w, w2, d, z, te.ACT_SILU, g, db, ws, dx, dw)
        copies = [t.clone() for t in bufs[1][:4]]
    for _ in range(3):
        for t in bufs[1]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(want, copies))
    G.check_no_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,K,outs", [("bf16", 1, 512, ("y", "res")), ("fp8", 24, 512, ("z", "y", "q")),
                                           ("mxfp8", 24, 4096, ("z", "q")), ("nvfp4", 300, 512, ("y32", "res")),
                                           ("fp8", 300, 4096, ("z", "y", "q"))])
def test_streams_and_graphs(kind, T, K, outs):
    """The same bits on another stream and in a graph, call behind call."""
    o = forward(kind, T, K, 416, "gelu", outs + ("bias",))
    names = [n for n in ("z", "y", "q", "s", "amax") if o.get(n) is not None]
    get = lambda n: o[n].t if isinstance(o[n], Out) else o[n]   # noqa: E731
    want = [get(n).clone() for n in names]
    side = torch.cuda.Stream()
    for n in names:
        get(n).zero_()
    torch.cuda.synchronize()
    o["call"](side)
    side.synchronize()
    assert all(torch.equal(get(n), v) for n, v in zip(names, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            o["call"]()
    for _ in range(2):
        for n in names:
            get(n).zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(get(n), v) for n, v in zip(names, want))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24, 100, 300])
def test_a_block_of_calls_waits_for_its_inputs(T):
    """Kernels are set up before what is in front of them in the stream has ended: norm, up projection and down
    projection onto the residual stream, whose input comes late by a copy or by an event from another stream, give the
    bits that they give one call at a time; eagerly and in a graph."""
    K, Fc = 512, 2560
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(T, K, generator=g).bfloat16().to(G.DEV) for _ in range(4)]
    w1, w2 = (torch.randn(*s, generator=g).mul(0.06).to(G.DEV) for s in ((Fc, K), (K, Fc)))
    gamma, beta, b1, b2, one = (torch.ones(K, device=G.DEV), torch.zeros(K, device=G.DEV), torch.ones(Fc, device=G.DEV),
                                torch.ones(K, device=G.DEV), G.scalar(1.0))
    w16, w8, v8 = w1.bfloat16(), *((w * 64).to(torch.float8_e4m3fn).view(torch.uint8) for w in (w1, w2))
    x, y, out = torch.zeros_like(xs[0]), torch.empty_like(xs[0]), torch.empty_like(xs[0])
    q, hq, amax, qamax = G.u8(T, K), G.u8(T, Fc), G.scalar(), G.scalar()
    h16 = torch.empty(T, Fc, dtype=torch.bfloat16, device=G.DEV)
    side, late = torch.cuda.Stream(), torch.zeros(64 << 20, device=G.DEV)

    def chain(i, how):
        if how == "event":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                late.add_(1.0)                                  # some 0.1 ms before x arrives
                x.copy_(xs[i])
            torch.cuda.current_stream().wait_stream(side)
        else:
            late.add_(1.0)
            x.copy_(xs[i])
        te.te_add_layernorm_fp8(x, gamma, beta, 1e-5, te.E4M3, one, q, y=y, amax_out=qamax)
        te.te_act_gemm_bf16(y, w16, te.ACT_GELU, y=h16, bias=b1)
        te.te_act_gemm_fp8(q, te.E4M3, w8, te.E4M3, one, one, te.ACT_GELU, bias=b1, q=hq, q_scale=one, q_amax=amax)
        te.te_act_gemm_fp8(hq, te.E4M3, v8, te.E4M3, one, one, te.ACT_NONE, bias=b2, residual=x, y=out)
        x.zero_()                                               # and nothing reads x afterwards
        return [t.clone() for t in (y, h16, hq, out, amax, qamax)]

    want = []
    for i in range(4):
        want.append(chain(i, "copy"))
        torch.cuda.synchronize()
    for how in ("event", "copy"):
        got = [chain(i % 4, how) for i in range(12)]
        torch.cuda.synchronize()
        for i, outs in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 4])), (how, i)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [chain(i, how) for i in range(4)]
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for i, outs in enumerate(got):
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), (how, i, "graph")


# ---- refusals: nothing reaches the GPU -------------------------------------------------------------

def test_wrapper_refusals():
    bf = torch.bfloat16
    x, w, y = torch.zeros(4, 32, dtype=bf), torch.zeros(64, 32, dtype=bf), torch.zeros(4, 64, dtype=bf)
    for bad in ((x[0], w), (x, torch.zeros(64, 16, dtype=bf))):                  # shapes
        with pytest.raises(ValueError):
            te.te_act_gemm_bf16(*bad, te.ACT_GELU, y=y)
    with pytest.raises(ValueError):                                               # not on the GPU
        te.te_act_gemm_bf16(x, w, te.ACT_GELU, y=y)
    with pytest.raises(TypeError):                                                # dtype of y
        te.te_act_gemm_bf16(x, w, te.ACT_GELU, y=y.half())
    with pytest.raises(TypeError):                                                # z is bf16
        te.te_act_gemm_bf16(x, w, te.ACT_GELU, z=y.float())
    with pytest.raises((TypeError, ValueError)):                                  # a residual of another type than y
        te.te_act_gemm_bf16(x, w, te.ACT_GELU, y=y.float(), residual=y)
    with pytest.raises(ValueError):
        te.te_act_dgrad_fp8(x.to(torch.uint8), te.E5M2, w[:, :16].to(torch.uint8), te.E4M3, None, None, y, 0, y)
    with pytest.raises(ValueError):
        te.te_act_bwd_bf16(x, w, w, x[0], y, 0, y)
    with pytest.raises(TypeError):                                                # z is needed for an activation
        te.te_act_bwd_bf16(x, w, w, x, None, te.ACT_GELU, y)


def test_library_refusals():
    import ctypes
    L = te.lib()
    ok, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)     # never dereferenced

    def bf(x=ok, w=ok, bias=None, act=te.ACT_GELU, res=None, z=None, y=ok, dt=te.BF16, T=4, K=32, N=32):
        return L.te_act_gemm_bf16(x, w, bias, act, res, z, y, dt, T, K, N, None)

    assert bf(K=24) == 2 and bf(N=24) == 2 and bf(K=0) == 2 and bf(N=0) == 2 and bf(T=-1) == 2
    assert bf(act=4) == 8 and bf(act=-1) == 8 and bf(dt=te.E4M3) == 4
    assert bf(y=None) == 1 and bf(x=None) == 1 and bf(w=None) == 1 and bf(y=None, z=ok, res=ok) == 1
    for name in ("x", "w", "bias", "res", "z", "y"):
        assert bf(**{name: odd}) == 3
    assert bf(T=0, x=None, w=None, y=None) == 0

    def f8(fx=te.E4M3, y=ok, res=None, q=None, qf=te.E4M3, sc=None, am=None, inv=None, si=ok, T=4):
        return L.te_act_gemm_fp8(ok, fx, ok, te.E4M3, si, ok, None, 0, res, None, y, te.BF16, q, qf, sc, am, inv, T, 32, 32, None)

    assert f8(fx=te.BF16) == 4 and f8(q=ok, sc=ok, qf=te.E2M1) == 4 and f8(q=ok, sc=ok, res=ok) == 5
    assert f8(si=None) == 1 and f8(q=ok) == 1 and f8(am=ok) == 1 and f8(inv=ok) == 1 and f8(y=None) == 1
    assert f8(q=odd, sc=ok) == 3 and f8(T=0) == 0 and f8(T=0, inv=ok) == 1

    def mx(sx=ok, q=None, s=None, K=32, N=32):
        return L.te_act_gemm_mxfp8(ok, te.E4M3, sx, ok, te.E4M3, ok, None, 0, None, None, ok, te.BF16, q, s, 4, K, N, None)

    assert mx(K=48) == 2 and mx(N=24) == 2 and mx(q=ok, s=ok, N=48) == 2 and mx(q=ok) == 1 and mx(s=ok) == 1
    assert mx(sx=None) == 1 and mx(sx=odd) == 3 and mx(q=ok, s=odd) == 3

    def nv(g=ok, y=ok, K=32, N=32):
        return L.te_act_gemm_nvfp4(ok, ok, g, ok, ok, ok, None, 0, None, None, y, te.BF16, 4, K, N, None)

    assert nv(K=16) == 2 and nv(N=24) == 2 and nv(g=None) == 1 and nv(y=None) == 1
    need = te.te_act_dbias_workspace_bytes(4, 32)
    assert need == 32 * 4 and te.te_act_dbias_workspace_bytes(33, 32) == 2 * 32 * 4 and te.te_act_dbias_workspace_bytes(0, 32) == 0

    def dg(fd=te.E5M2, z=ok, act=0, dz=ok, db=None, ws=None, n=0, si=ok):
        return L.te_act_dgrad_fp8(ok, fd, ok, te.E4M3, ok, si, z, act, dz, db, ws, n, 4, 32, 32, None)

    assert dg(dz=None) == 1 and dg(si=None) == 1 and dg(z=None) == 1 and dg(fd=te.E8M0) == 4 and dg(z=odd) == 3
    assert dg(db=ok) == 1 and dg(db=ok, ws=ok, n=need - 1) == 2 and dg(db=ok, ws=odd, n=need) == 3
    assert dg(db=ctypes.c_void_p(0x1002), ws=ok, n=need) == 3 and dg(act=7) == 8
    assert L.te_act_dgrad_mxfp8(ok, te.E4M3, ok, ok, te.E4M3, ok, ok, 0, ok, None, None, 0, 4, 32, 48, None) == 2
    assert L.te_act_dgrad_nvfp4(ok, ok, ok, ok, ok, ok, odd, 0, ok, None, None, 0, 4, 32, 32, None) == 3

    def bwd(x=ok, w=ok, dx=ok, dw=ok, dt=te.BF16, acc=0, K=32, dz=ok):
        return L.te_act_bwd_bf16(x, w, ok, ok, ok, 0, dz, None, None, 0, dx, dw, dt, acc, 4, K, 32, 32, None)

    assert bwd(K=24) == 2 and bwd(dt=te.E4M3) == 4 and bwd(acc=1) == 4 and bwd(acc=2) == 8
    assert bwd(x=None) == 1 and bwd(w=None) == 1 and bwd(dz=None) == 1 and bwd(dx=odd) == 3 and bwd(dw=odd) == 3
