"""The stage-by-stage check of the gated block on a block that the oracle computes: it accepts it under every
recipe, and it rejects mistakes planted there that a comparison of norms lets through."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import quantize as Q
from oracle.gated import act, act_grad, gated, gated_bwd
from oracle.rmsnorm import rmsnorm, rmsnorm_bwd
from tests.gated_stages import GRAD, _values, verify

T, K, FC = 32, 64, 128
RECIPES = ["bf16", "fp8_delayed", "mxfp8"]


def bf(v):
    return F.bf16_bits_to_f32(F.f64_to_bf16_bits(np.asarray(v, np.float64))).astype(np.float64)


def oracle_block(recipe, mistake=None):
    rng = np.random.default_rng(4)
    n = rng.standard_normal
    t = dict(gamma=(1 + 0.1 * n(K)).astype(np.float32).astype(np.float64), w=bf(n((2 * FC, K)) * K ** -0.5),
             w2=bf(n((K, FC)) * FC ** -0.5), x=bf(n((T, K))), res=bf(n((T, K))), dout=bf(n((T, K)) * 1e-3),
             dr=bf(n((T, K)) * 1e-3), row={}, col={}, srow={}, scol={}, scale={}, inv={})

    def quantize(name, v, row=True, col=True):
        fmt = "e5m2" if name in GRAD else "e4m3"
        v = np.asarray(v, np.float32)
        if recipe == "mxfp8":
            if row:
                t["row"][name], t["srow"][name] = Q.mxfp8_quantize(v)
            if col:
                t["col"][name], t["scol"][name] = Q.mxfp8_quantize(np.ascontiguousarray(v.T))
            return
        if name not in t["scale"]:
            s = np.float32({"e4m3": 448, "e5m2": 57344}[fmt] / np.abs(v).max())
            t["scale"][name], t["inv"][name] = s, np.float32(1) / s
        if row:
            t["row"][name] = Q.fp8_cast(v, t["scale"][name], fmt)
        if col:
            t["col"][name] = Q.fp8_cast(np.ascontiguousarray(v.T), t["scale"][name], fmt)

    plain = recipe == "bf16"

    def row(name):
        return t[name] if plain else _values(t, name, False, recipe)

    def col(name):
        return t[name].T if plain else _values(t, name, True, recipe)

    r, y, rs = rmsnorm(t["x"], t["gamma"], 1e-5, t["res"])
    t["r"], t["y"], t["rsigma"] = bf(r), bf(y), rs
    if not plain:
        for name in ("w", "w2", "dout"):
            quantize(name, t[name])
        quantize("y", y, col=False)
        quantize("y", t["y"], row=False)
    h, g, u = gated(row("y"), row("w"), "silu")
    t["gu"], t["h"] = bf(np.concatenate([g, u], 1)), bf(h)
    if not plain:
        quantize("h", h, col=False)
        quantize("h", t["h"], row=False)
    t["out"] = bf(row("h") @ row("w2").T)
    t["dw2"] = bf(col("dout") @ col("h").T)
    g, u = t["gu"][:, :FC], t["gu"][:, FC:]
    dg, du = gated_bwd(row("dout"), col("w2").T, g, u, "silu")
    if mistake == "slope":                        # act' without its second term
        dg = (row("dout") @ col("w2").T) * u / (1 + np.exp(-g))
    t["dgu"] = bf(np.concatenate([dg, du], 1))
    if not plain:
        quantize("dgu", t["dgu"])
    t["dy"], t["dw"] = bf(row("dgu") @ col("w").T), bf(col("dgu") @ col("y").T)
    dx, t["dgamma"] = rmsnorm_bwd(t["dy"], t["r"], t["gamma"], t["rsigma"], t["dr"])
    t["dx"] = bf(dx)
    return t


@pytest.mark.parametrize("recipe", RECIPES)
def test_the_oracles_block_passes(recipe):
    verify(oracle_block(recipe), recipe)


@pytest.mark.parametrize("recipe", RECIPES)
def test_mistakes_are_rejected(recipe):
    def rejected(t):
        with pytest.raises(AssertionError):
            verify(t, recipe)

    rejected(oracle_block(recipe, "slope"))
    good = oracle_block(recipe)
    rejected({**good, "dx": good["dr"]})                                   # the block's own gradient dropped
    for name in ("out", "gu", "h", "dgu", "dy", "dx", "dw", "dw2", "dgamma", "y", "r", "rsigma"):
        for factor in (0.5, 1.5, 1.02, 0.0):
            rejected({**good, name: good[name] * factor})
    for name in ("out", "dw", "dw2", "dy"):
        part = good[name].copy()
        part[:, -part.shape[1] // 3:] = 0                                  # a third of the columns missing
        rejected({**good, name: part})
    if recipe != "bf16":
        for copies in ("row", "col"):
            for name in good[copies]:
                q = good[copies][name].copy()
                q[3] = q[4]
                rejected({**good, copies: {**good[copies], name: q}})
    if recipe == "fp8_delayed":
        for name in good["inv"]:
            rejected({**good, "inv": {**good["inv"], name: good["inv"][name] * np.float32(1.25)}})
