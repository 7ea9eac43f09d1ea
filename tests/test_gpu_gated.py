"""The gated projections (every operand kind, activation and output) and their backward passes,
against the 64-bit oracle on the operands' own values.

Tolerances.  A product over K terms is within K 2^-23 S of the exact one, S the sum of the terms'
sizes (fp32 accumulation, whatever its order); the activation's exponential is within
(2 + 1.2 |z|) 2^-23 relative and its sigmoid within (8 + 4 |z|) 2^-23 with the rounding of z;
an output of half a step r (bf16 2^-8, E4M3 2^-4, E5M2 2^-3) adds r of the value.
"""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from oracle import formats as F
from oracle import quantize as Q
from oracle.gated import act, act_grad, gated, gated_bwd
from tests import gpu_util as G

E23 = 2.0 ** -23
BF = 2.0 ** -8
ACT = {"silu": te.ACT_SILU, "gelu": te.ACT_GELU}
FMT = {"e4m3": te.E4M3, "e5m2": te.E5M2}
HALF = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
SMALL = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}


def _tiles(s, mult):
    """Logical scale bytes [R, C] -> the tensor-core layout, padding zero."""
    R, C = s.shape
    p = np.zeros((-(-R // 128) * 128, -(-C // mult) * mult), np.uint8)
    p[:R, :C] = s
    r, c = p.shape
    return p.reshape(r // 128, 4, 32, c // 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(G.DEV)


class Operand:
    """A quantized operand: device tensors, and its values in 64 bits."""

    def __init__(self, a, kind, fmt="e4m3"):
        a = np.asarray(a, np.float32)
        self.fmt = fmt
        if kind == "bf16":
            self.q = torch.from_numpy(a).bfloat16().to(G.DEV)
            self.v = self.q.cpu().double().numpy()
        elif kind == "fp8":
            scale = np.float32(FMAX[fmt] / np.abs(a).max())
            q = Q.fp8_cast(a, scale, fmt)
            self.q, self.inv = _dev(q), G.scalar(float(np.float32(1) / scale))
            self.v = F.decode(q, fmt).astype(np.float64) * self.inv.item()
        elif kind == "mxfp8":
            q, s = Q.mxfp8_quantize(a)
            self.q, self.s, self.v = _dev(q), _dev(_tiles(s, 4)), Q.mxfp8_dequant(q, s)
        else:
            q, s, g = Q.nvfp4_quantize(a, Q.amax(a))
            self.q, self.s, self.g = _dev(Q.pack_e2m1(q)), _dev(_tiles(s, 16)), G.scalar(float(g))
            self.v = Q.nvfp4_dequant(q, s, g)


class Out:
    """An output tensor inside a poisoned buffer, so that a write past its end shows."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        n = int(np.prod(shape))
        self.n = n
        self.buf = torch.full((n + 4096,), 119, dtype=dtype, device=G.DEV)
        self.t = self.buf[:n].view(*shape)

    def np(self):
        assert bool((self.buf[self.n:] == 119).all()), "wrote past the end"
        return self.t.detach().cpu().double().numpy() if self.t.dtype != torch.uint8 else self.t.cpu().numpy()


def _sizes(g, u, dg, du, kind):
    """|h|'s error before its rounding, from the errors dg, du of g and u."""
    z = np.abs(g) if kind == "silu" else 2 * np.abs(g) * (1 + 0.05 * g * g)
    a = np.abs(act(g, kind)) + 1.2 * dg
    return 1.2 * dg * (np.abs(u) + du) + a * du + (8 + 4 * z) * E23 * a * (np.abs(u) + du)


def _codes(q, v, err, fmt, what):
    got = F.decode(q, fmt).astype(np.float64)
    c = np.clip(v, -FMAX[fmt], FMAX[fmt])
    tol = np.maximum(HALF[fmt] * (np.abs(c) + err), SMALL[fmt]) + err
    assert np.all(np.abs(got - c) <= tol), (what, float(np.max(np.abs(got - c) / tol)))


def _inputs(T, K, Fc, seed):
    rng = np.random.default_rng(seed + T + 3 * K + 7 * Fc)
    return rng.standard_normal((T, K)), rng.standard_normal((2 * Fc, K)) * (1.5 / np.sqrt(K))


def _forward(kind, T, K, Fc, actk, outs, seed=0, fmt="e4m3", stream=None, xw=None):
    a, b = _inputs(T, K, Fc, seed)
    x, w = xw or (Operand(a, kind), Operand(b, kind))
    o = dict(h=Out(T, Fc) if "h" in outs else None, gu=Out(T, 2 * Fc) if "gu" in outs else None)
    t = {k: v.t if v else None for k, v in o.items()}
    A = ACT[actk]
    if kind == "bf16":
        te.te_gated_gemm_bf16(x.q, w.q, A, stream=stream, **t)
    elif kind == "fp8":
        more = {}
        if "q" in outs:
            o["q"], o["amax"], o["inv"] = Out(T, Fc, dtype=torch.uint8), G.scalar(-1.0), G.scalar(-1.0)
            o["scale"] = np.float32(FMAX[fmt] / 3.0)                     # larger values saturate
            more = dict(q_h=o["q"].t, h_fmt=FMT[fmt], h_scale=G.scalar(float(o["scale"])), h_amax=o["amax"],
                        h_scale_inv=o["inv"])
        te.te_gated_gemm_fp8(x.q, te.E4M3, w.q, te.E4M3, x.inv, w.inv, A, stream=stream, **t, **more)
    elif kind == "mxfp8":
        more = {}
        if "q" in outs:
            o["q"] = Out(T, Fc, dtype=torch.uint8)
            o["s"] = Out(te.te_scale_bytes(te.E8M0, T, Fc), dtype=torch.uint8)
            more = dict(q_h=o["q"].t, s_h=o["s"].t)
        te.te_gated_gemm_mxfp8(x.q, x.s, w.q, w.s, A, stream=stream, **t, **more)
    else:
        te.te_gated_gemm_nvfp4(x.q, x.s, x.g, w.q, w.s, w.g, A, stream=stream, **t)
    torch.cuda.synchronize()
    G.check_no_device_error()
    return x, w, o


def _check_forward(kind, T, K, Fc, actk, outs, fmt="e4m3", xw=None):
    x, w, o = _forward(kind, T, K, Fc, actk, outs, fmt=fmt, xw=xw)
    h64, g64, u64 = gated(x.v, w.v, actk)
    S = np.abs(x.v) @ np.abs(w.v).T * ((K + 4) * E23)
    dg, du = S[:, :Fc], S[:, Fc:]
    err = _sizes(g64, u64, dg, du, actk)
    if o["gu"]:
        gu, want = o["gu"].np(), np.concatenate([g64, u64], 1)
        assert np.all(np.abs(gu - want) <= BF * (np.abs(want) + S) + S), "gu"
    if o["h"]:
        assert np.all(np.abs(o["h"].np() - h64) <= BF * (np.abs(h64) + err) + err), "h"
    if "q" in o and kind == "fp8":
        sc = float(o["scale"])
        _codes(o["q"].np(), h64 * sc, err * sc + np.abs(h64) * sc * E23, fmt, "q")
        assert abs(o["amax"].item() - np.abs(h64).max()) <= err.max()
        assert np.float32(o["inv"].item()) == np.float32(1) / o["scale"]
    elif "q" in o:
        raw = o["s"].np()
        s = te.te_scale_unswizzle(te.E8M0, T, Fc, raw).astype(np.int64)
        top = np.abs(h64).reshape(T, -1, 32)
        slack = err.reshape(T, -1, 32)
        lo = np.floor(np.log2((top - slack).max(-1).clip(1e-30))) + 119
        hi = np.floor(np.log2((top + slack).max(-1))) + 119
        assert np.all((s >= lo) & (s <= hi)), "scales"
        assert int(raw.astype(np.int64).sum()) == int(s.sum()), "padding"
        mul = np.exp2(127.0 - np.repeat(s, 32, 1))
        _codes(o["q"].np(), h64 * mul, err * mul, "e4m3", "q")


# one token to several tiles of tokens; widths that end inside a box, a tile, a k-step
GENERAL = [(1, 16, 16), (1, 208, 272), (2, 80, 48), (15, 64, 112), (17, 400, 144), (33, 768, 256), (127, 48, 128),
           (129, 320, 400), (256, 64, 144), (257, 96, 1040), (385, 128, 64)]
BLOCK = [(1, 32, 128), (3, 96, 256), (31, 416, 128), (64, 256, 384), (129, 160, 128), (300, 544, 640)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", GENERAL)
@pytest.mark.parametrize("actk,outs", [("silu", "h"), ("gelu", ("h", "gu")), ("silu", "gu")])
def test_bf16(T, K, Fc, actk, outs):
    _check_forward("bf16", T, K, Fc, actk, (outs,) if isinstance(outs, str) else outs)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", GENERAL)
@pytest.mark.parametrize("actk,outs,fmt", [("silu", ("q",), "e4m3"), ("gelu", ("h", "gu", "q"), "e5m2"),
                                           ("silu", ("h",), "e4m3")])
def test_fp8(T, K, Fc, actk, outs, fmt):
    _check_forward("fp8", T, K, Fc, actk, outs, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", BLOCK)
@pytest.mark.parametrize("kind,actk,outs", [("mxfp8", "silu", ("q",)), ("mxfp8", "gelu", ("h", "gu", "q")),
                                            ("nvfp4", "silu", ("h",)), ("nvfp4", "gelu", ("h", "gu"))])
def test_block_scaled(T, K, Fc, kind, actk, outs):
    _check_forward(kind, T, K, Fc, actk, outs)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,outs", [("bf16", ("h", "gu")), ("fp8", ("h", "gu", "q")), ("mxfp8", ("h", "gu", "q")),
                                       ("nvfp4", ("h", "gu"))])
def test_several_tiles_per_cta(kind, outs):
    """More tiles than CTA pairs: the rings, the accumulators and the staging boxes are used again."""
    _check_forward(kind, 2100 if kind in ("bf16", "fp8") else 2080, 128, 1664, "silu", outs)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", [(1, 4096, 2480), (8, 2064, 80), (9, 1040, 1232), (16, 4112, 32), (24, 4096, 48),
                                    (32, 2096, 1248), (25, 4096, 32), (20, 4096, 80), (40, 128, 10000), (64, 2064, 272),
                                    (31, 6000, 16), (3, 16400, 32)])
@pytest.mark.parametrize("kind,outs,fmt", [("bf16", ("h", "gu"), "e4m3"), ("fp8", ("h", "gu", "q"), "e4m3"),
                                           ("fp8", ("q",), "e5m2")])
def test_few_tokens(T, K, Fc, kind, outs, fmt):
    """Long rows and more units of columns than SMs: the streaming kernels' steps, their prefetch
    across units and the reuse of their rings and exchange buffers."""
    _check_forward(kind, T, K, Fc, "gelu", outs, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", [(1, 4128, 1280), (8, 8256, 128), (5, 160, 4992), (2, 64, 2560), (9, 4128, 128),
                                    (7, 13696, 128)])
@pytest.mark.parametrize("kind,actk,outs", [("mxfp8", "silu", ("q",)), ("mxfp8", "gelu", ("h", "gu", "q")),
                                            ("mxfp8", "silu", ("gu",)), ("nvfp4", "gelu", ("h", "gu"))])
def test_few_tokens_block_scaled(T, K, Fc, kind, actk, outs):
    """Several steps of the streaming kernels, more runs of columns than SMs, and lengths past what they hold."""
    _check_forward(kind, T, K, Fc, actk, outs)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("fx,fw", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_mxfp8_operand_formats(T, fx, fw):
    a, b = _inputs(T, 224, 128, 5)
    ops = []
    for v, f in ((a, fx), (b, fw)):
        q, sc = Q.mxfp8_quantize(v.astype(np.float32), f)
        ops.append((_dev(q), _dev(_tiles(sc, 4)), Q.mxfp8_dequant(q, sc, f)))
    (x, sx, xv), (w, sw, wv) = ops
    h = Out(T, 128)
    te.te_gated_gemm_mxfp8(x, sx, w, sw, te.ACT_SILU, h=h.t, fx=FMT[fx], fw=FMT[fw])
    torch.cuda.synchronize()
    h64, g64, u64 = gated(xv, wv, "silu")
    S = np.abs(xv) @ np.abs(wv).T * (228 * E23)
    err = _sizes(g64, u64, S[:, :128], S[:, 128:], "silu")
    assert np.all(np.abs(h.np() - h64) <= BF * (np.abs(h64) + err) + err)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 40, 200])
@pytest.mark.parametrize("fx,fw", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_fp8_operand_formats(T, fx, fw):
    a, b = _inputs(T, 208, 144, 5)
    x, w = Operand(a, "fp8", fx), Operand(b, "fp8", fw)
    h = Out(T, 144)
    te.te_gated_gemm_fp8(x.q, FMT[fx], w.q, FMT[fw], x.inv, w.inv, te.ACT_SILU, h=h.t)
    torch.cuda.synchronize()
    h64, g64, u64 = gated(x.v, w.v, "silu")
    S = np.abs(x.v) @ np.abs(w.v).T * (212 * E23)
    err = _sizes(g64, u64, S[:, :144], S[:, 144:], "silu")
    assert np.all(np.abs(h.np() - h64) <= BF * (np.abs(h64) + err) + err)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_special_values_stay_in_their_row(T):
    a, b = _inputs(T, 64, 160, 1)
    a[T // 2, 3] = np.nan
    x, w = Operand(a, "bf16"), Operand(b, "bf16")
    x, w, o = _forward("bf16", T, 64, 160, "silu", ("h", "gu"), xw=(x, w))
    h = o["h"].np()
    assert np.isnan(h[T // 2]).all() and np.isfinite(np.delete(h, T // 2, 0)).all()
    # saturated gates: act(g) -> g and -> 0, no NaN from the exponential's overflow
    a, b = np.full((T, 16), 8.0), np.ones((32, 16))
    b[:8] = -1.0                                              # gate rows 0-7: g = -128, rows 8-15: g = 128; u = 128
    x, w, o = _forward("bf16", T, 16, 16, "gelu", ("h",), xw=(Operand(a, "bf16"), Operand(b, "bf16")))
    h = o["h"].np()
    assert np.all(np.abs(h[:, :8]) <= 1e-30) and np.all(h[:, 8:] == 16384.0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 200])
def test_fp8_amax_keeps_nan_and_ignores_the_ragged_edge(T):
    """F = 16: three quarters of the last box belong to the up projection's rows, which must not
    reach the amax; a NaN code must."""
    a, b = _inputs(T, 32, 16, 2)
    b[16:] *= 50.0                                            # u rows large: u * act(u) would dominate
    x, w = Operand(a, "fp8"), Operand(b, "fp8")
    _check_forward("fp8", T, 32, 16, "silu", ("q",), xw=(x, w))
    x.q[T - 1, 5] = 0x7F
    _, _, o = _forward("fp8", T, 32, 16, "silu", ("q",), xw=(x, w))
    assert np.isnan(o["amax"].item()) and np.all(o["q"].np()[T - 1] & 0x7F == 0x7F)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 70, 200])
def test_rows_past_the_last_token_stay_out(T):
    """A weight that is not finite makes the tile's rows past the last token NaN (zero times infinity):
    they reach neither the amax nor the padding of the scales."""
    a, b = _inputs(T, 64, 128, 4)
    x, w = Operand(np.abs(a) + 0.1, "fp8"), Operand(b, "fp8", "e5m2")
    w.q[5, 7] = 0x7C                                           # +inf in a gate row: g = +inf, h = +-inf
    h, q, amax = Out(T, 128), Out(T, 128, dtype=torch.uint8), G.scalar(-1.0)
    te.te_gated_gemm_fp8(x.q, te.E4M3, w.q, te.E5M2, x.inv, w.inv, te.ACT_SILU, h=h.t, q_h=q.t, h_scale=G.scalar(1.0),
                         h_amax=amax)
    torch.cuda.synchronize()
    assert np.isinf(h.np()[:, 5]).all() and np.isfinite(np.delete(h.np(), 5, 1)).all()
    assert np.isposinf(amax.item())
    x, w = Operand(a, "mxfp8"), Operand(b, "mxfp8")
    w.q[5, 7] = 0x7F                                           # NaN
    q, s = Out(T, 128, dtype=torch.uint8), Out(te.te_scale_bytes(te.E8M0, T, 128), dtype=torch.uint8)
    te.te_gated_gemm_mxfp8(x.q, x.s, w.q, w.s, te.ACT_SILU, q_h=q.t, s_h=s.t)
    torch.cuda.synchronize()
    raw = s.np()
    assert int(raw.astype(np.int64).sum()) == int(te.te_scale_unswizzle(te.E8M0, T, 128, raw).astype(np.int64).sum())


@pytest.mark.gpu
def test_no_tokens():
    w = torch.zeros(64, 32, dtype=torch.bfloat16, device=G.DEV)
    x = torch.zeros(0, 32, dtype=torch.bfloat16, device=G.DEV)
    te.te_gated_gemm_bf16(x, w, te.ACT_SILU, h=torch.zeros(0, 32, dtype=torch.bfloat16, device=G.DEV))
    amax, inv, one = G.scalar(-1.0), G.scalar(-1.0), G.scalar(1.0)
    te.te_gated_gemm_fp8(x.to(torch.uint8), te.E4M3, w.to(torch.uint8), te.E4M3, one, one, te.ACT_SILU,
                         q_h=torch.zeros(0, 32, dtype=torch.uint8, device=G.DEV), h_scale=G.scalar(4.0), h_amax=amax,
                         h_scale_inv=inv)
    gu, dy, w2 = (torch.zeros(*s, dtype=torch.bfloat16, device=G.DEV) for s in ((0, 64), (0, 16), (16, 32)))
    dw = torch.ones(64, 32, device=G.DEV)
    te.te_gated_bwd_bf16(x, w, w2, dy, gu, te.ACT_SILU, gu.clone(), dx=x.clone(), dw=dw, accumulate=1)
    torch.cuda.synchronize()
    assert amax.item() == 0 and inv.item() == 0.25 and bool((dw == 1).all())
    te.te_gated_bwd_bf16(x, w, w2, dy, gu, te.ACT_SILU, gu.clone(), dw=dw)
    torch.cuda.synchronize()
    assert not dw.any()


# ---- backward -----------------------------------------------------------------------------------

def _check_dgu(dgu, dy_v, w2_v, gu, actk, N):
    Fc = gu.shape[1] // 2
    g, u = gu[:, :Fc], gu[:, Fc:]
    dg64, du64 = gated_bwd(dy_v, w2_v, g, u, actk)
    ddh = np.abs(dy_v) @ np.abs(w2_v) * ((N + 4) * E23)
    dh = np.abs(dy_v @ w2_v) + ddh
    z = np.abs(g) if actk == "silu" else 2 * np.abs(g) * (1 + 0.05 * g * g)
    f = (12 + 4 * z) * E23
    slope = np.abs(act_grad(g, actk)) + f * (1 + np.abs(g) * (1 if actk == "silu" else 1.6 * (1 + 0.14 * g * g)))
    a = np.abs(act(g, actk)) * (1 + f)
    for got, want, err in ((dgu[:, :Fc], dg64, np.abs(u) * (ddh * slope + dh * (slope - np.abs(act_grad(g, actk)) + 4 * E23 * slope))),
                           (dgu[:, Fc:], du64, ddh * a + dh * a * f)):
        tol = BF * (np.abs(want) + err) + err + 1e-38
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


def _bwd_inputs(T, Fc, N, seed=0):
    rng = np.random.default_rng(seed + T + 5 * Fc + 11 * N)
    gu = torch.from_numpy(rng.standard_normal((T, 2 * Fc)) * 1.5).bfloat16().to(G.DEV)
    return rng.standard_normal((T, N)) * 1e-3, rng.standard_normal((N, Fc)) * 0.05, gu


def _dgrad(kind, T, Fc, N, actk, gu=None, dgu=None):
    dy, w2, gu_ = _bwd_inputs(T, Fc, N)
    gu = gu_ if gu is None else gu
    d, w = Operand(dy, kind, "e5m2"), Operand(w2.T, kind)
    o = Out(T, 2 * Fc) if dgu is None else None
    t = o.t if o else dgu
    if kind == "fp8":
        te.te_gated_dgrad_fp8(d.q, te.E5M2, w.q, te.E4M3, d.inv, w.inv, gu, ACT[actk], t)
    elif kind == "mxfp8":
        te.te_gated_dgrad_mxfp8(d.q, d.s, w.q, w.s, gu, ACT[actk], t)
    else:
        te.te_gated_dgrad_nvfp4(d.q, d.s, d.g, w.q, w.s, w.g, gu, ACT[actk], t)
    torch.cuda.synchronize()
    G.check_no_device_error()
    return d, w, gu, o


@pytest.mark.gpu
@pytest.mark.parametrize("T,Fc,N", [(1, 16, 32), (3, 272, 96), (33, 144, 64), (128, 48, 160), (130, 400, 64),
                                    (257, 1040, 32), (2100, 2640, 64)])
@pytest.mark.parametrize("kind,actk", [("fp8", "silu"), ("fp8", "gelu"), ("mxfp8", "silu"), ("nvfp4", "gelu")])
def test_dgrad(T, Fc, N, kind, actk):
    d, w, gu, o = _dgrad(kind, T, Fc, N, actk)
    _check_dgu(o.np(), d.v, w.v.T, gu.cpu().double().numpy(), actk, N)


@pytest.mark.gpu
def test_dgrad_in_place():
    _, _, gu, o = _dgrad("fp8", 300, 400, 64, "silu")
    same = gu.clone()
    _dgrad("fp8", 300, 400, 64, "silu", gu=same, dgu=same)
    assert torch.equal(same, o.t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc,N", [(1, 16, 16, 16), (3, 208, 272, 80), (33, 64, 144, 48), (100, 768, 128, 768),
                                      (129, 80, 400, 64), (257, 96, 1040, 32), (1001, 48, 80, 112),
                                      (70, 96, 784, 1552), (1700, 304, 1600, 1600), (300, 400, 3200, 64),
                                      (2100, 2304, 2560, 1600)])
@pytest.mark.parametrize("actk,dwt", [("silu", torch.bfloat16), ("gelu", torch.float32)])
def test_bwd_bf16(T, K, Fc, N, actk, dwt):
    dy, w2, gu = _bwd_inputs(T, Fc, N)
    a, b = _inputs(T, K, Fc, 3)
    x, w, d, w2 = (Operand(v, "bf16") for v in (a, b, dy, w2))
    dgu, dx, dw = Out(T, 2 * Fc), Out(T, K), Out(2 * Fc, K, dtype=dwt)
    te.te_gated_bwd_bf16(x.q, w.q, w2.q, d.q, gu, ACT[actk], dgu.t, dx.t, dw.t)
    torch.cuda.synchronize()
    got = dgu.np()
    _check_dgu(got, d.v, w2.v, gu.cpu().double().numpy(), actk, N)
    # dx and dw from the dgu that was written
    for out, want, size, n, half in ((dx, got @ w.v, np.abs(got) @ np.abs(w.v), 2 * Fc, BF),
                                     (dw, got.T @ x.v, np.abs(got).T @ np.abs(x.v), T, BF if dwt is torch.bfloat16 else E23)):
        tol = half * np.abs(want) + (n + 4) * E23 * (1 + half) * size + 1e-38
        assert np.all(np.abs(out.np() - want) <= tol)
    if dwt is torch.float32:
        first = dw.t.clone()
        te.te_gated_bwd_bf16(x.q, w.q, w2.q, d.q, gu, ACT[actk], dgu.t, dw=dw.t, accumulate=1)
        torch.cuda.synchronize()
        assert torch.equal(dw.t, first + first)
    G.check_no_device_error()


@pytest.mark.gpu
def test_streams_graphs_and_repeats():
    """The same bits on another stream, in a graph, and again."""
    x, w, o = _forward("fp8", 300, 256, 400, "silu", ("h", "gu", "q"))
    side = torch.cuda.Stream()
    _, _, p = _forward("fp8", 300, 256, 400, "silu", ("h", "gu", "q"), stream=side, xw=(x, w))
    for k in ("h", "gu", "q"):
        assert torch.equal(o[k].t, p[k].t)
    assert torch.equal(o["amax"], p["amax"])
    h = torch.zeros_like(o["h"].t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        te.te_gated_gemm_fp8(x.q, te.E4M3, w.q, te.E4M3, x.inv, w.inv, te.ACT_SILU, h=h)
    for _ in range(2):
        h.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, o["h"].t)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24, 300])
def test_calls_set_up_early_wait_for_their_inputs(T):
    """Kernels are set up before what is in front of them in the stream has ended: a chain of norm, gated
    projections (all kinds of kernels) and a copy, whose input comes late, by an event, from another
    stream, from a copy or a memset, gives the bits that it gives one call at a time; eagerly and in a graph."""
    K, Fc = 512, 1280
    g = torch.Generator().manual_seed(3)
    xs = [torch.randn(T, K, generator=g).bfloat16().to(G.DEV) for _ in range(4)]
    w = torch.randn(2 * Fc, K, generator=g).mul(0.06).to(G.DEV)
    gamma, w16, one = torch.ones(K, device=G.DEV), w.bfloat16(), G.scalar(1.0)
    w8 = (w * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    x, y = torch.zeros_like(xs[0]), torch.empty_like(xs[0])
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
        elif how == "copy":
            late.add_(1.0)
            x.copy_(xs[i])
        else:
            x.copy_(xs[i])
            late.zero_()
        te.te_rmsnorm_fp8(x, gamma, 1e-5, te.E4M3, one, q, y=y, amax_out=qamax)
        te.te_gated_gemm_bf16(y, w16, te.ACT_SILU, h=h16)
        te.te_gated_gemm_fp8(q, te.E4M3, w8, te.E4M3, one, one, te.ACT_SILU, q_h=hq, h_scale=one, h_amax=amax)
        x.zero_()                                               # and nothing reads x afterwards
        return [t.clone() for t in (y, h16, hq, amax, qamax)]

    want = []
    for i in range(4):
        want.append(chain(i, "plain"))
        torch.cuda.synchronize()
    for how in ("plain", "event", "copy"):
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


# contractions long enough for a tile to be shared by two or four CTA pairs, with few tiles (four), more
# (two), ragged edges, and parts of unequal length
# and a last, partial wave behind full ones
SHARED = [(70, 3216, 16), (100, 3200, 144), (129, 4112, 272), (300, 6160, 1600), (513, 3216, 400), (65, 8208, 128),
          (2100, 3216, 1280), (1300, 6160, 2048)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", SHARED)
@pytest.mark.parametrize("kind,actk,outs,fmt", [("bf16", "silu", ("h", "gu"), "e4m3"), ("fp8", "gelu", ("h", "gu", "q"), "e4m3"),
                                                ("fp8", "silu", ("q",), "e5m2")])
def test_shared_contraction(T, K, Fc, kind, actk, outs, fmt):
    _check_forward(kind, T, K, Fc, actk, outs, fmt)
    # and the same bits every time
    x, w, o = _forward(kind, T, K, Fc, actk, outs, fmt=fmt)
    _, _, p = _forward(kind, T, K, Fc, actk, outs, fmt=fmt, xw=(x, w))
    for k in ("h", "gu", "q"):
        if o.get(k):
            assert torch.equal(o[k].t, p[k].t)


@pytest.mark.gpu
@pytest.mark.parametrize("T,Fc,N", [(1, 16, 3216), (70, 272, 3200), (300, 144, 4112), (300, 2640, 6160)])
@pytest.mark.parametrize("actk", ["silu", "gelu"])
def test_shared_contraction_dgrad(T, Fc, N, actk):
    d, w, gu, o = _dgrad("fp8", T, Fc, N, actk)
    _check_dgu(o.np(), d.v, w.v.T, gu.cpu().double().numpy(), actk, N)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc,N", [(1001, 768, 2048, 768), (60, 64, 1040, 2048), (3000, 1024, 1024, 256),
                                      (2100, 2304, 2560, 1600)])
def test_bwd_overlap_and_graph(T, K, Fc, N):
    """dX and dW overlap and start while dGU's kernel drains: twenty calls in a row, eager and in a
    graph, give the bits that calls on their own give, and what follows in the stream sees both."""
    dy, w2, gu = _bwd_inputs(T, Fc, N, 6)
    a, b = _inputs(T, K, Fc, 6)
    x, w, d, w2 = (torch.from_numpy(v).bfloat16().to(G.DEV) for v in (a, b, dy, w2))
    bufs = [(torch.empty(T, 2 * Fc, dtype=torch.bfloat16, device=G.DEV), torch.empty_like(x), torch.empty_like(w))
            for _ in range(2)]

    def call(scale, i):
        g, dx, dw = bufs[i]
        te.te_gated_bwd_bf16(x, w, w2, d * scale, gu, te.ACT_SILU, g, dx=dx, dw=dw)
        return g.clone(), dx.clone(), dw.clone()

    want = []
    for i in range(20):
        want.append(call(2.0 ** (i % 3), 0))
        torch.cuda.synchronize()
    got = [call(2.0 ** (i % 3), i % 2) for i in range(20)]
    torch.cuda.synchronize()
    for p, q in zip(want, got):
        assert all(torch.equal(m, n) for m, n in zip(p, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g, dx, dw = bufs[1]
        for i in range(5):
            te.te_gated_bwd_bf16(x, w, w2, d, gu, te.ACT_SILU, g, dx=dx, dw=dw)
        copies = [t.clone() for t in bufs[1]]
    for _ in range(3):
        for t in bufs[1]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(want[0], copies))
    G.check_no_device_error()


# ---- refusals: nothing reaches the GPU -------------------------------------------------------------

def test_wrapper_refusals():
    bf = torch.bfloat16
    x, w, h = torch.zeros(4, 32, dtype=bf), torch.zeros(64, 32, dtype=bf), torch.zeros(4, 32, dtype=bf)
    for bad in ((x[0], w), (x, w[:63]), (x, torch.zeros(64, 16, dtype=bf))):     # shapes
        with pytest.raises(ValueError):
            te.te_gated_gemm_bf16(*bad, te.ACT_SILU, h=h)
    with pytest.raises(ValueError):                                               # not on the GPU
        te.te_gated_gemm_bf16(x, w, te.ACT_SILU, h=h)
    with pytest.raises(TypeError):                                                # dtype
        te.te_gated_gemm_bf16(x.half(), w, te.ACT_SILU, h=h)
    with pytest.raises(ValueError):                                               # a strided view
        te.te_gated_gemm_bf16(torch.zeros(32, 4, dtype=bf).t(), w, te.ACT_SILU, h=h)
    with pytest.raises(ValueError):
        te.te_gated_dgrad_fp8(x.to(torch.uint8), te.E5M2, w[:, :16].to(torch.uint8), te.E4M3, None, None, h, 0, h)
    with pytest.raises(ValueError):
        te.te_gated_bwd_bf16(x, w, w, x[0], h, 0, h)


def test_library_refusals():
    import ctypes
    L = te.lib()
    ok, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)     # never dereferenced

    def bf(x=ok, w=ok, act=0, h=ok, gu=None, T=4, K=32, Fc=32):
        return L.te_gated_gemm_bf16(x, w, act, h, gu, T, K, Fc, None)

    assert bf(K=24) == 2 and bf(Fc=24) == 2 and bf(K=0) == 2 and bf(Fc=0) == 2 and bf(T=-1) == 2
    assert bf(act=2) == 8 and bf(act=-1) == 8
    assert bf(h=None) == 1 and bf(x=None) == 1 and bf(w=None) == 1
    assert bf(x=odd) == 3 and bf(w=odd) == 3 and bf(h=odd) == 3 and bf(gu=odd) == 3
    assert bf(T=0, x=None, w=None, h=None) == 0

    def f8(fx=te.E4M3, h=ok, q=None, qf=te.E4M3, sc=None, am=None, inv=None, si=ok, T=4):
        return L.te_gated_gemm_fp8(ok, fx, ok, te.E4M3, si, ok, 0, h, None, q, qf, sc, am, inv, T, 32, 32, None)

    assert f8(fx=te.BF16) == 4 and f8(q=ok, sc=ok, qf=te.E2M1) == 4
    assert f8(si=None) == 1 and f8(q=ok) == 1 and f8(am=ok) == 1 and f8(inv=ok) == 1 and f8(h=None) == 1
    assert f8(q=odd, sc=ok) == 3 and f8(T=0) == 0 and f8(T=0, inv=ok) == 1

    def mx(sx=ok, q=None, s=None, K=32, Fc=128):
        return L.te_gated_gemm_mxfp8(ok, te.E4M3, sx, ok, te.E4M3, ok, 0, ok, None, q, s, 4, K, Fc, None)

    assert mx(K=48) == 2 and mx(Fc=64) == 2 and mx(q=ok) == 1 and mx(s=ok) == 1 and mx(sx=None) == 1 and mx(sx=odd) == 3

    def nv(g=ok, h=ok, K=32, Fc=128):
        return L.te_gated_gemm_nvfp4(ok, ok, g, ok, ok, ok, 0, h, None, 4, K, Fc, None)

    assert nv(K=16) == 2 and nv(Fc=144) == 2 and nv(g=None) == 1 and nv(h=None) == 1
    assert L.te_gated_dgrad_fp8(ok, te.E5M2, ok, te.E4M3, ok, ok, ok, 0, None, 4, 32, 32, None) == 1
    assert L.te_gated_dgrad_fp8(ok, te.E5M2, ok, te.E4M3, ok, None, ok, 0, ok, 4, 32, 32, None) == 1
    assert L.te_gated_dgrad_fp8(ok, te.E8M0, ok, te.E4M3, ok, ok, ok, 0, ok, 4, 32, 32, None) == 4
    assert L.te_gated_dgrad_mxfp8(ok, te.E4M3, ok, ok, te.E4M3, ok, ok, 0, ok, 4, 32, 48, None) == 2
    assert L.te_gated_dgrad_nvfp4(ok, ok, ok, ok, ok, ok, odd, 0, ok, 4, 32, 32, None) == 3

    def bwd(x=ok, w=ok, dx=ok, dw=ok, dt=te.BF16, acc=0, K=32, dgu=ok):
        return L.te_gated_bwd_bf16(x, w, ok, ok, ok, 0, dgu, dx, dw, dt, acc, 4, K, 32, 32, None)

    assert bwd(K=24) == 2 and bwd(dt=te.E4M3) == 4 and bwd(acc=1) == 4 and bwd(acc=2) == 8
    assert bwd(x=None) == 1 and bwd(w=None) == 1 and bwd(dgu=None) == 1 and bwd(dx=odd) == 3 and bwd(dw=odd) == 3


def _twice(kind, T, K, Fc, actk, outs, fmt="e4m3"):
    """The outputs of a second call on the same operands are the first's, bit for bit."""
    x, w, o = _forward(kind, T, K, Fc, actk, outs, fmt=fmt)
    _, _, p = _forward(kind, T, K, Fc, actk, outs, fmt=fmt, xw=(x, w))
    for name in ("h", "gu", "q", "s", "amax"):
        a, b = o.get(name), p.get(name)
        if a is not None:
            a, b = (a.t, b.t) if isinstance(a, Out) else (a, b)
            assert torch.equal(a, b), name


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", [(9, 4112, 16), (13, 2064, 512), (33, 4112, 1040), (64, 2048, 2048), (27, 4096, 2576),
                                    (62, 528, 4864), (63, 528, 4880), (1, 4608, 1536), (7, 8208, 1088), (12, 16400, 80),
                                    (65, 4112, 1040), (128, 2048, 2576), (101, 8208, 80), (90, 4112, 4864),
                                    (90, 4112, 4880)])
@pytest.mark.parametrize("kind,actk,outs,fmt", [("bf16", "silu", ("h", "gu"), "e4m3"),
                                                ("fp8", "gelu", ("h", "gu", "q"), "e5m2")])
def test_few_tokens_shared_contraction(T, K, Fc, kind, actk, outs, fmt):
    """Few columns on a long row: 2, 4 or 8 CTAs share it, with parts of unequal length, a ragged last
    k-tile, tokens that end inside a group of four, and the sizes on both sides of the rule."""
    _check_forward(kind, T, K, Fc, actk, outs, fmt)
    _twice(kind, T, K, Fc, actk, outs, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,Fc", [(1, 320, 128), (3, 1056, 256), (6, 2080, 1024), (30, 4128, 2048), (64, 2048, 4096),
                                    (33, 8224, 128), (61, 800, 9728), (40, 800, 9856), (65, 4128, 1280), (128, 8224, 256),
                                    (99, 4128, 384), (79, 4128, 640), (81, 2080, 640)])
@pytest.mark.parametrize("kind,actk,outs", [("mxfp8", "silu", ("h", "gu", "q")), ("nvfp4", "gelu", ("h", "gu"))])
def test_few_tokens_shared_contraction_block_scaled(T, K, Fc, kind, actk, outs):
    _check_forward(kind, T, K, Fc, actk, outs)
    _twice(kind, T, K, Fc, actk, outs)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [10, 42, 74])
def test_shared_contraction_keeps_what_is_not_finite_in_its_row_and_column(T):
    a, b = _inputs(T, 4096, 256, 8)
    x, w = Operand(np.abs(a) + 0.1, "fp8"), Operand(b, "fp8", "e5m2")
    w.q[5, 3000] = 0x7C                                        # +inf in a gate row
    h, q, amax = Out(T, 256), Out(T, 256, dtype=torch.uint8), G.scalar(-1.0)
    te.te_gated_gemm_fp8(x.q, te.E4M3, w.q, te.E5M2, x.inv, w.inv, te.ACT_SILU, h=h.t, q_h=q.t, h_scale=G.scalar(1.0),
                         h_amax=amax)
    torch.cuda.synchronize()
    assert np.isinf(h.np()[:, 5]).all() and np.isfinite(np.delete(h.np(), 5, 1)).all() and np.isposinf(amax.item())
    x, w = Operand(a, "mxfp8"), Operand(b, "mxfp8")
    x.q[T - 1, 100] = 0x7F                                     # NaN
    h, q = Out(T, 256), Out(T, 256, dtype=torch.uint8)
    s = Out(te.te_scale_bytes(te.E8M0, T, 256), dtype=torch.uint8)
    te.te_gated_gemm_mxfp8(x.q, x.s, w.q, w.s, te.ACT_SILU, h=h.t, q_h=q.t, s_h=s.t)
    torch.cuda.synchronize()
    assert np.isnan(h.np()[T - 1]).all() and np.isfinite(h.np()[:T - 1]).all()
    raw = s.np()
    assert int(raw.astype(np.int64).sum()) == int(te.te_scale_unswizzle(te.E8M0, T, 256, raw).astype(np.int64).sum())
