"""The gated projections by the kernel that a call takes: every form with several tiles a CTA and several
k-tiles a tile, the rasters of long contractions, and sums that only a full fp32 accumulator carries.

Each case names the form that it is for and asks the captured launch whether it is the one, so that a
change of the rule that picks the kernel cannot leave a form without its test.  Tolerances are those
of the comparisons in test_gpu_gated (counted roundings); the sums of integers are compared for
equality."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G
from tests.kernel_names import form
from tests.test_gpu_gated import ACT, Out, _check_dgu, _check_forward, _dev, _tiles

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


class Codes:
    """A quantized operand from codes and scales as given, and its values in 64 bits.  `v`: the codes'
    values [R, C], `s`: the blocks' scales (a block is 32 in MXFP8, 16 in NVFP4)."""

    def __init__(self, kind, v, s=None, factor=1.0):
        R, C = v.shape
        t = torch.from_numpy(np.ascontiguousarray(v, np.float32))
        if kind == "bf16":
            self.q = t.bfloat16().to(G.DEV)
            self.v = self.q.cpu().double().numpy()
            return
        if kind == "nvfp4":
            n = np.searchsorted(E2M1[:8], np.abs(v)).astype(np.uint8) | ((v < 0) * 8).astype(np.uint8)
            self.q = _dev(n[:, 0::2] | (n[:, 1::2] << 4))
            self.v = E2M1[n]
            sb = torch.from_numpy(s.astype(np.float32)).to(F8)
            self.s, self.g = _dev(_tiles(sb.view(torch.uint8).numpy(), 16)), G.scalar(factor)
            self.v = self.v * np.repeat(sb.double().numpy(), 16, 1) * self.g.item()
            return
        c = t.to(F8)
        self.q, self.v = c.view(torch.uint8).to(G.DEV), c.double().numpy()
        if kind == "fp8":
            self.inv = G.scalar(factor)
            self.v = self.v * self.inv.item()
        else:
            e = np.log2(s).astype(np.int64)
            self.s = _dev(_tiles((e + 127).astype(np.uint8), 4))
            self.v = self.v * np.repeat(np.exp2(e), 32, 1)


def _random(kind, R, C, rng, size):
    """Values of about `size` (root mean square)."""
    if kind == "bf16":
        return Codes(kind, rng.standard_normal((R, C), np.float32) * size)
    if kind == "fp8":
        return Codes(kind, rng.standard_normal((R, C), np.float32) * 40, None, size / 40)
    if kind == "mxfp8":
        e = rng.integers(-2, 3, (R, C // 32)) + int(np.round(np.log2(size / 40)))
        return Codes(kind, rng.standard_normal((R, C), np.float32) * 40, np.exp2(e.astype(np.float64)))
    return Codes(kind, E2M1[rng.integers(0, 16, (R, C))], rng.uniform(0.5, 4.0, (R, C // 16)), size / 5.0)


def _operands(kind, T, K, F):
    rng = np.random.default_rng(T + 3 * K + 7 * F)
    return _random(kind, T, K, rng, 1.0), _random(kind, 2 * F, K, rng, 1.5 / np.sqrt(K))


def _form(kind, x, w, T, F):
    h = torch.empty(T, F, dtype=torch.bfloat16, device=G.DEV)
    act = te.ACT_SILU

    def call(stream):
        if kind == "bf16":
            te.te_gated_gemm_bf16(x.q, w.q, act, h=h, stream=stream)
        elif kind == "fp8":
            te.te_gated_gemm_fp8(x.q, te.E4M3, w.q, te.E4M3, x.inv, w.inv, act, h=h, stream=stream)
        elif kind == "mxfp8":
            te.te_gated_gemm_mxfp8(x.q, x.s, w.q, w.s, act, h=h, stream=stream)
        else:
            te.te_gated_gemm_nvfp4(x.q, x.s, x.g, w.q, w.s, w.g, act, h=h, stream=stream)

    call(None)
    return form(call)


def _n_tiles(kind, T, F, what):
    if what == "pair":
        return -(-T // 256) * -(-F // 128)
    return -(-F // (64 if kind in ("bf16", "fp8") else 128))


OUTS = {"bf16": ("h", "gu"), "fp8": ("h", "gu", "q"), "mxfp8": ("h", "gu", "q"), "nvfp4": ("h", "gu")}

# the streams with one CTA a tile, two and three tiles a CTA: the ring, the accumulators and (BF16, FP8) the
# exchange of g and u are used again
STREAM = [(k, T, K, F) for k in ("bf16", "fp8")
          for T, K, F in [(9, 528, 10000), (24, 4112, 10000), (32, 528, 16400), (24, 272, 20016), (33, 2064, 10000),
                          (64, 4112, 10000), (64, 2064, 20016)]]
STREAM += [(k, T, K, F) for k in ("mxfp8", "nvfp4")
           for T, K, F in [(3, 416, 19584), (32, 2080, 19584), (24, 288, 39040), (33, 1056, 19584), (64, 4128, 19584)]]


@pytest.mark.parametrize("kind,T,K,F", STREAM)
def test_streams_with_several_tiles_per_cta(kind, T, K, F):
    x, w = _operands(kind, T, K, F)
    _check_forward(kind, T, K, F, "gelu", OUTS[kind], "e4m3", (x, w))
    what, ctas = _form(kind, x, w, T, F)
    assert what == "stream" and ctas < _n_tiles(kind, T, F, what), (what, ctas)


# pairs with several tiles each and more k-tiles than stages (the second tile walks K backwards), and the
# raster from 64 k-tiles on, with either side longer
PAIR = [(k, 2080, 2080, 1664) for k in ("bf16", "fp8", "mxfp8", "nvfp4")]
PAIR += [("fp8", 300, 8224, 5136), ("mxfp8", 300, 8224, 5120), ("nvfp4", 300, 16416, 5120), ("fp8", 10300, 8224, 272),
         ("mxfp8", 10300, 8224, 256), ("nvfp4", 10300, 16416, 256)]


@pytest.mark.parametrize("kind,T,K,F", PAIR)
def test_pairs_with_several_tiles_of_several_k_tiles(kind, T, K, F):
    x, w = _operands(kind, T, K, F)
    _check_forward(kind, T, K, F, "silu", OUTS[kind], "e4m3", (x, w))
    what, ctas = _form(kind, x, w, T, F)
    assert what == "pair" and ctas // 2 < _n_tiles(kind, T, F, what), (what, ctas)


def _dgrad(kind, d, w, gu, act, dgu, stream=None):
    if kind == "fp8":
        te.te_gated_dgrad_fp8(d.q, te.E4M3, w.q, te.E4M3, d.inv, w.inv, gu, act, dgu, stream=stream)
    elif kind == "mxfp8":
        te.te_gated_dgrad_mxfp8(d.q, d.s, w.q, w.s, gu, act, dgu, stream=stream)
    else:
        te.te_gated_dgrad_nvfp4(d.q, d.s, d.g, w.q, w.s, w.g, gu, act, dgu, stream=stream)


@pytest.mark.parametrize("kind,T,F,N", [(k, 2100, 2640, 2080) for k in ("fp8", "mxfp8", "nvfp4")] +
                         [("fp8", 300, 10256, 8208), ("mxfp8", 300, 10256, 8224), ("nvfp4", 300, 10256, 16416),
                          ("fp8", 10300, 272, 8208), ("mxfp8", 10300, 272, 8224), ("nvfp4", 10300, 272, 16416)])
def test_dgrad_with_several_tiles_of_several_k_tiles(kind, T, F, N):
    rng = np.random.default_rng(T + F + N)
    d, w = _random(kind, T, N, rng, 1e-3), _random(kind, F, N, rng, 0.05)
    gu = torch.from_numpy(rng.standard_normal((T, 2 * F)) * 1.5).bfloat16().to(G.DEV)
    o = Out(T, 2 * F)
    _dgrad(kind, d, w, gu, ACT["gelu"], o.t)
    torch.cuda.synchronize()
    _check_dgu(o.np(), d.v, w.v.T, gu.cpu().double().numpy(), "gelu", N)
    what, ctas = form(lambda s: _dgrad(kind, d, w, gu, ACT["gelu"], o.t, s))
    assert what == "pair" and ctas // 2 < -(-T // 256) * -(-F // 256), (what, ctas)
    G.check_no_device_error()


# ---- sums in full ------------------------------------------------------------------------------

def _integers(kind, R, K, rng, sign):
    """Rows whose products with one another have a large part that comes and goes -- 256 a term over the
    first half of K and (one operand: `sign`) -256 over the second -- and a few small integers in
    the first, the middle and the last 32 columns.  K = 32 (2 n + 1)."""
    n = K // 32
    small = np.zeros(n, bool)
    small[[0, n // 2, n - 1]] = True
    flip = np.where(np.arange(n) > n // 2, -1.0, 1.0) if sign else np.ones(n)
    low = rng.integers(-3, 4, (R, K)) if sign else rng.integers(0, 4, (R, K))
    low = low * (rng.random((R, K)) < 0.5)
    per = 16 if kind == "nvfp4" else 32
    sm = np.repeat(small, 32)[None, :]
    scale = {"bf16": 1.0, "fp8": 1.0, "mxfp8": 16.0, "nvfp4": 4.0}[kind]
    v = np.where(sm, low, np.repeat(flip, 32)[None, :] * (16.0 / scale))
    s = np.repeat(np.where(small, 1.0, scale), 32 // per)[None, :].repeat(R, 0)
    return Codes(kind, v, s)


EXACT = [("bf16", 1, 4128, 1024, "decode"), ("bf16", 30, 1056, 256, "decode"), ("bf16", 24, 4128, 512, "stream shared"),
         ("bf16", 64, 4128, 512, "stream shared"), ("bf16", 100, 8224, 512, "stream shared"),
         ("bf16", 24, 4128, 10112, "stream"), ("bf16", 300, 4128, 512, "pair shared"), ("bf16", 300, 4128, 10240, "pair"),
         ("fp8", 1, 4128, 1024, "decode"), ("fp8", 16, 1056, 256, "decode"), ("fp8", 24, 4128, 512, "stream shared"),
         ("fp8", 64, 4128, 512, "stream shared"), ("fp8", 100, 8224, 512, "stream shared"),
         ("fp8", 24, 4128, 10112, "stream"), ("fp8", 300, 4128, 512, "pair shared"), ("fp8", 300, 8224, 5120, "pair")]
EXACT += [(k, T, K, F, f) for k in ("mxfp8", "nvfp4")
          for T, K, F, f in [(1, 4128, 512, "stream shared"), (24, 4128, 512, "stream shared"),
                             (64, 8224, 512, "stream shared"), (100, 8224, 512, "stream shared"),
                             (24, 2080, 19584, "stream"), (300, 4128, 10240, "pair")]]


@pytest.mark.parametrize("kind,T,K,F,what", EXACT)
def test_sums_of_integers_are_exact(kind, T, K, F, what):
    """The partial sums grow to 2^17 to 2^20 beside units that must survive: an accumulator, or an exchange of
    parts, of fewer than 17 to 20 bits would lose them.  g and u themselves are at most 256: exact in bf16."""
    rng = np.random.default_rng(T + K + F)
    x, w = _integers(kind, T, K, rng, False), _integers(kind, 2 * F, K, rng, True)
    want = x.v @ w.v.T
    assert np.abs(want).max() <= 256 and np.abs(x.v[0] * w.v[0]).sum() >= 2 ** 17
    gu = Out(T, 2 * F)
    if kind == "bf16":
        te.te_gated_gemm_bf16(x.q, w.q, te.ACT_SILU, gu=gu.t)
    elif kind == "fp8":
        te.te_gated_gemm_fp8(x.q, te.E4M3, w.q, te.E4M3, x.inv, w.inv, te.ACT_SILU, gu=gu.t)
    elif kind == "mxfp8":
        te.te_gated_gemm_mxfp8(x.q, x.s, w.q, w.s, te.ACT_SILU, gu=gu.t)
    else:
        te.te_gated_gemm_nvfp4(x.q, x.s, x.g, w.q, w.s, w.g, te.ACT_SILU, gu=gu.t)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(gu.np(), want)
    assert _form(kind, x, w, T, F)[0] == what
    G.check_no_device_error()


@pytest.mark.parametrize("kind", ["fp8", "mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,F,what", [(100, 256, "shared"), (300, 10256, "")])
def test_dgrad_sums_of_integers_are_exact(kind, T, F, what):
    """At g = 128, u = 1 the sigmoid is 1, so dg = dh and du = 128 dh."""
    rng = np.random.default_rng(T + F)
    d, w = _integers(kind, T, 4128, rng, False), _integers(kind, F, 4128, rng, True)
    dh = d.v @ w.v.T
    gu = torch.ones(T, 2 * F, dtype=torch.bfloat16, device=G.DEV)
    gu[:, :F] = 128.0
    o = Out(T, 2 * F)
    _dgrad(kind, d, w, gu, te.ACT_SILU, o.t)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(o.np(), np.concatenate([dh, 128 * dh], 1))
    got = form(lambda s: _dgrad(kind, d, w, gu, te.ACT_SILU, o.t, s))[0]
    assert got == ("pair shared" if what and kind == "fp8" else "pair")
