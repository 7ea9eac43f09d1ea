"""The gated block checked stage by stage: every kernel's output against the 64-bit result of the tensors that
the kernel itself read (the quantized copies with their scales, the stored bf16 tensors), so that each
comparison is as tight as one rounding, and every copy against the oracle's quantization of its
source, bit for bit.

``verify(t, recipe)``: t maps names to arrays -- gamma, w, w2, x, res, dout, dr, r, y, rsigma, gu, h, out, dgu, dy,
dx, dw, dw2, dgamma in 64 bits; for the quantized recipes row[name] and col[name], codes, with
srow / scol (logical scales, MXFP8) or scale / inv (fp32 numbers, FP8)."""
import numpy as np

from oracle import formats as F
from oracle import quantize as Q
from oracle.gated import act, act_grad, gated, gated_bwd
from oracle.rmsnorm import rmsnorm, rmsnorm_bwd

E = 2.0 ** -24
E23 = 2.0 ** -23
BF = 2.0 ** -8
E4 = 2.0 ** -4
GRAD = ("dout", "dgu")


def _near(got, want, err, what, half=BF):
    """One rounding of a value that is itself within `err` of `want`."""
    tol = half * (np.abs(want) + err) + err + 1e-38
    bad = np.abs(got - want) / tol
    assert np.all(bad <= 1), (what, float(np.nanmax(bad)))


def _product(got, a, b, what):
    """A bf16 product a b^T: fp32 sums of K terms, then one rounding."""
    S = np.abs(a) @ np.abs(b).T * ((a.shape[1] + 4) * E23)
    _near(got, a @ b.T, S, what)


def _fmt(t, name, recipe):
    return "e5m2" if recipe == "fp8_delayed" and name in GRAD else "e4m3"


def _values(t, name, col, recipe):
    """The values of a copy, scales included."""
    q = (t["col"] if col else t["row"])[name]
    if recipe == "mxfp8":
        return Q.mxfp8_dequant(q, (t["scol"] if col else t["srow"])[name])
    return F.decode(q, _fmt(t, name, recipe)).astype(np.float64) * float(t["inv"][name])


def _copy(t, name, col, recipe):
    """The copy is the oracle's quantization of the tensor, bit for bit."""
    src = np.ascontiguousarray(t[name].T if col else t[name]).astype(np.float32)
    q = (t["col"] if col else t["row"])[name]
    if recipe == "mxfp8":
        want, s = Q.mxfp8_quantize(src)
        assert np.array_equal((t["scol"] if col else t["srow"])[name], s), (name, col, "scales")
    else:
        want = Q.fp8_cast(src, t["scale"][name], _fmt(t, name, recipe))
        assert np.float32(t["inv"][name]) == np.float32(1) / np.float32(t["scale"][name])
    assert np.array_equal(q, want), (name, "col" if col else "row")


def _fused(t, name, ideal, err, recipe):
    """A row copy that the kernel cast from its fp32 value (within `err` of `ideal`): half a step of E4M3."""
    q = F.decode(t["row"][name], "e4m3").astype(np.float64)
    if recipe == "mxfp8":
        s = t["srow"][name].astype(np.int64)
        top, off = (np.abs(v).reshape(v.shape[0], -1, 32) for v in (ideal, np.broadcast_to(err, ideal.shape)))
        lo, hi = (np.floor(np.log2((top + k * off).max(-1).clip(1e-300))) + 119 for k in (-1, 1))
        assert np.all((s >= np.maximum(lo, 0)) & (s <= np.maximum(hi, 0))), (name, "scales")
        mul = np.exp2(127.0 - np.repeat(s, 32, 1))
    else:
        mul = float(t["scale"][name])
    c = np.clip(ideal * mul, -448, 448)
    e = err * mul + 2 * E * np.abs(c)
    assert np.all(np.abs(q - c) <= np.maximum(E4 * (np.abs(c) + e), 2.0 ** -10) + e), name


def verify(t, recipe):
    plain = recipe == "bf16"
    T, K = t["x"].shape
    Fc = t["w2"].shape[1]
    # the norm
    s64, y64, rs64 = rmsnorm(t["x"], t["gamma"], 1e-5, t["res"])
    _near(t["r"], s64, E * np.abs(s64), "r")
    assert np.all(np.abs(t["rsigma"] - rs64) <= 40 * E * rs64), "rsigma"
    _near(t["y"], y64, 46 * E * np.abs(y64), "y")
    if not plain:
        _fused(t, "y", y64, 46 * E * np.abs(y64), recipe)
        for n in ("w", "w2", "dout", "dgu"):
            _copy(t, n, False, recipe)
        for n in ("w", "w2", "dout", "dgu", "y", "h"):
            _copy(t, n, True, recipe)

    def row(n):
        return t[n] if plain else _values(t, n, False, recipe)

    def col(n):
        return t[n].T if plain else _values(t, n, True, recipe)

    # the gated projections
    y, w = row("y"), row("w")
    h64, g64, u64 = gated(y, w, "silu")
    S = np.abs(y) @ np.abs(w).T * ((K + 4) * E23)
    dg, du = S[:, :Fc], S[:, Fc:]
    a = np.abs(act(g64, "silu")) + 1.2 * dg
    err = 1.2 * dg * (np.abs(u64) + du) + a * du + (8 + 4 * np.abs(g64)) * E23 * a * (np.abs(u64) + du)
    _near(t["gu"], np.concatenate([g64, u64], 1), S, "gu")
    _near(t["h"], h64, err, "h")
    if not plain:
        _fused(t, "h", h64, err, recipe)
    _product(t["out"], row("h"), row("w2"), "out")
    # backward
    _product(t["dw2"], col("dout"), col("h"), "dw2")
    g, u = t["gu"][:, :Fc], t["gu"][:, Fc:]
    d, w2 = row("dout"), col("w2").T                       # w2 [K, F]
    dg64, du64 = gated_bwd(d, w2, g, u, "silu")
    ddh = np.abs(d) @ np.abs(w2) * ((K + 4) * E23)
    dh, f = np.abs(d @ w2) + ddh, (12 + 4 * np.abs(g)) * E23
    slope, av = np.abs(act_grad(g, "silu")), np.abs(act(g, "silu")) * (1 + f)
    more = f * (1 + np.abs(g)) + 4 * E23 * (slope + f * (1 + np.abs(g)))
    _near(t["dgu"][:, :Fc], dg64, np.abs(u) * (ddh * (slope + more) + dh * more), "dg")
    _near(t["dgu"][:, Fc:], du64, ddh * av + dh * av * f, "du")
    _product(t["dy"], row("dgu"), col("w"), "dy")
    _product(t["dw"], col("dgu"), col("y"), "dw")
    dx64, dgamma64 = rmsnorm_bwd(t["dy"], t["r"], t["gamma"], t["rsigma"], t["dr"])
    xhat, p = np.abs(t["r"] * t["rsigma"][:, None]), np.abs(t["dy"] * t["gamma"])
    size = t["rsigma"][:, None] * (p + xhat * (p * xhat).mean(1, keepdims=True))
    _near(t["dx"], dx64, 72 * E * size + E * np.abs(dx64), "dx")
    assert np.all(np.abs(t["dgamma"] - dgamma64) <= (T + 4) * E * (np.abs(t["dy"]) * xhat).sum(0)), "dgamma"
