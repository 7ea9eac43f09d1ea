"""The linear with bias, activation and residual by the kernel that a call takes: every form with several tiles a CTA and
several k-tiles a tile, sums that only a full fp32 accumulator carries, cut into segments or not, and first calls inside a
stream capture.

Each case names the form that it is for and asks the captured launch whether it is the one, so that a change of the rule
that picks the kernel cannot leave a form without its test.  Tolerances are those of test_gpu_act; the sums of integers
are compared for equality."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G
from tests.kernel_names import launched
from tests.test_gpu_act import check_dz, check_forward, dgrad, forward, same_again
from tests.test_gpu_gated import Out
from tests.test_gpu_gated_forms import _integers, _random

pytestmark = pytest.mark.gpu


def form(call):
    """'decode', 'stream', 'stream shared', 'pair' or 'pair shared' ('shared': several CTAs or pairs have a tile's K),
    and the CTAs of the grid."""
    for name, ctas in launched(call):
        if "act_decode_kernel" in name:
            return "decode", ctas
        m = re.search(r"act_stream_kernelILi\d+ELi\d+ELb([01])E", name) or re.search(r"gemm_kernelILi\d+ELi\d+ELi[34]ELb([01])E", name)
        if m:
            return ("stream" if "stream" in name else "pair") + (" shared" if m[1] == "1" else ""), ctas
    raise AssertionError("no kernel of the linear was launched")


OUTS = {"bf16": ("z", "y", "bias"), "fp8": ("z", "y", "q", "bias"), "mxfp8": ("z", "y", "q", "bias"), "nvfp4": ("z", "y", "bias")}

# tokens, K, N and the form; tiles of the streams (128 x 32, 64 or 128 tokens) and of the pairs (256 x 256) past the SMs
FORMS = [(k, T, K, N, f) for k in ("bf16", "fp8")
         for T, K, N, f in [(1, 2064, 2064, "decode"), (3, 4112, 160, "decode"), (8, 1040, 1616, "decode"),
                            (8, 272, 8208, "stream shared"), (24, 528, 20016, "stream"), (33, 272, 40016, "stream"),
                            (100, 528, 20016, "stream"), (24, 4112, 528, "stream shared"), (64, 4112, 2064, "stream shared"),
                            (128, 4112, 528, "stream shared"), (200, 4112, 528, "stream shared"), (300, 528, 4112, "stream"),
                            (300, 1040, 16400, "stream"), (2080, 2080, 3344, "pair"), (2080, 8208, 272, "pair shared")]]
FORMS += [("bf16", 1100, 8208, 1040, "pair shared"), ("fp8", 1100, 8208, 1040, "stream")]
FORMS += [(k, T, K, N, f) for k in ("mxfp8", "nvfp4")
          for T, K, N, f in [(1, 4128, 544, "stream shared"), (24, 544, 20000, "stream"), (33, 288, 39040, "stream"),
                             (100, 544, 20000, "stream"), (64, 4128, 2080, "stream shared"), (200, 8224, 544, "stream shared"),
                             (300, 1056, 4128, "stream"), (2080, 2080, 3360, "pair"), (2500, 8224, 288, "pair")]]


def _operands(kind, T, K, N):
    rng = np.random.default_rng(T + 3 * K + 7 * N)
    return _random(kind, T, K, rng, 1.0), _random(kind, N, K, rng, 1.5 / np.sqrt(K))


@pytest.mark.parametrize("kind,T,K,N,what", FORMS)
def test_every_form(kind, T, K, N, what):
    x, w = _operands(kind, T, K, N)
    x.fmt = w.fmt = "e4m3"
    o = check_forward(kind, T, K, N, "gelu", OUTS[kind], ops=(x, w))
    same_again(o)
    assert form(o["call"])[0] == what
    o = check_forward(kind, T, K, N, "none", ("y32", "bias", "res"), ops=(x, w))
    same_again(o)
    assert form(o["call"])[0] == what


# ---- sums in full ------------------------------------------------------------------------------

EXACT = [(k, T, K, N, f) for k in ("bf16", "fp8")
         for T, K, N, f in [(1, 1056, 512, "decode"), (24, 4128, 512, "stream shared"), (64, 8224, 512, "stream shared"),
                            (24, 2080, 20000, "stream"), (200, 4128, 512, "stream shared"), (300, 1056, 4096, "stream"),
                            (2080, 8224, 272, "pair shared"), (2080, 4128, 3328, "pair")]]
EXACT += [(k, T, K, N, f) for k in ("mxfp8", "nvfp4")
          for T, K, N, f in [(1, 4128, 512, "stream shared"), (100, 8224, 512, "stream shared"), (24, 2080, 20000, "stream"),
                             (300, 1056, 4096, "stream"), (2080, 8224, 3328, "pair")]]


@pytest.mark.parametrize("yt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind,T,K,N,what", EXACT)
def test_sums_of_integers_are_exact(kind, T, K, N, what, yt):
    """The partial sums grow to 2^15 to 2^20 beside units that must survive: an accumulator, an exchange of parts or the
    sum of segments with fewer bits would lose them.  z itself is at most 256: exact in bf16."""
    rng = np.random.default_rng(T + K + N)
    x, w = _integers(kind, T, K, rng, False), _integers(kind, N, K, rng, True)
    want = x.v @ w.v.T
    assert np.abs(want).max() <= 256 and np.abs(x.v[0] * w.v[0]).sum() >= 2 ** 15
    y = Out(T, N, dtype=yt)

    def call(stream=None):
        kw = dict(y=y.t, stream=stream)
        if kind == "bf16":
            te.te_act_gemm_bf16(x.q, w.q, te.ACT_NONE, **kw)
        elif kind == "fp8":
            te.te_act_gemm_fp8(x.q, te.E4M3, w.q, te.E4M3, x.inv, w.inv, te.ACT_NONE, **kw)
        elif kind == "mxfp8":
            te.te_act_gemm_mxfp8(x.q, x.s, w.q, w.s, te.ACT_NONE, **kw)
        else:
            te.te_act_gemm_nvfp4(x.q, x.s, x.g, w.q, w.s, w.g, te.ACT_NONE, **kw)

    call()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(y.np(), want)
    assert form(call)[0] == what
    G.check_no_device_error()


@pytest.mark.parametrize("kind", ["fp8", "mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,F", [(100, 256), (300, 10256)])
def test_dgrad_sums_of_integers_are_exact(kind, T, F):
    """With a ReLU that lets every other token pass, dz is dh or zero; the sums of dz over tokens stay below 2^24."""
    rng = np.random.default_rng(T + F)
    d, w = _integers(kind, T, 8224, rng, False), _integers(kind, F, 8224, rng, True)
    d.fmt = "e4m3"
    on = (np.arange(T) % 2 == 0)[:, None]
    dh = d.v @ w.v.T * on
    z = torch.from_numpy(np.where(on, 1.0, -1.0).repeat(F, 1)).bfloat16().to(G.DEV)
    dz, db = Out(T, F), torch.full((F,), 7.0, device=G.DEV)
    kw = dict(dbias=db, workspace=torch.full((te.te_act_dbias_workspace_bytes(T, F) // 4,), float("nan"), device=G.DEV))
    if kind == "fp8":
        te.te_act_dgrad_fp8(d.q, te.E4M3, w.q, te.E4M3, d.inv, w.inv, z, te.ACT_RELU, dz.t, **kw)
    elif kind == "mxfp8":
        te.te_act_dgrad_mxfp8(d.q, d.s, w.q, w.s, z, te.ACT_RELU, dz.t, **kw)
    else:
        te.te_act_dgrad_nvfp4(d.q, d.s, d.g, w.q, w.s, w.g, z, te.ACT_RELU, dz.t, **kw)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(dz.np(), dh)
    np.testing.assert_array_equal(db.cpu().double().numpy(), dh.sum(0))
    G.check_no_device_error()


@pytest.mark.parametrize("kind,T,F,N", [("fp8", 2100, 2640, 2080), ("mxfp8", 2100, 2640, 2080), ("nvfp4", 2100, 2640, 2080),
                                        ("fp8", 300, 10256, 8208), ("mxfp8", 300, 10256, 8224), ("fp8", 10300, 272, 8208)])
def test_dgrad_with_several_tiles_of_several_k_tiles(kind, T, F, N):
    d, w, z, o, db = dgrad(kind, T, F, N, "gelu")
    check_dz(o.np(), db.cpu().double().numpy(), d.v, w.v.T, z.cpu().double().numpy(), "gelu", N)
    what, ctas = form(lambda s: dgrad(kind, T, F, N, "gelu", ops=(d, w), z=z, stream=s))
    assert what == "pair" and ctas // 2 < -(-T // 256) * -(-F // 256), (what, ctas)


def test_long_sums_in_fp32_do_not_shrink():
    """BF16, K = 16384: whole, the tensor cores' rounding towards zero leaves 1.9e-5 of the sums; in segments of 13
    k-tiles each is 13 x 4 additions long, 2^-24 of it at most each, and half of them on average: 8e-7 together here."""
    for T in (1, 24, 100, 300):
        o = forward("bf16", T, 16384, 512, "none", ("y32",))
        want = o["x"].v @ o["w"].v.T
        assert np.linalg.norm(o["y"].np() - want) <= 1e-6 * np.linalg.norm(want), T


def test_two_calls_at_once():
    """Calls on two streams at the same time, each with its own tensors, give the bits of calls on their own."""
    cases = [forward("bf16", 2000, 1024, 2048, "gelu", ("z", "y", "bias")), forward("mxfp8", 60, 4096, 1024, "gelu", ("z", "q", "bias")),
             forward("fp8", 2000, 1024, 2048, "relu", ("z", "y", "q"), seed=3), forward("nvfp4", 1, 2048, 2048, "none", ("y", "res"))]
    names = ("z", "y", "q", "s")
    want = [{n: o[n].t.clone() for n in names if o.get(n)} for o in cases]
    side = torch.cuda.Stream()
    for first in cases:
        for second in cases:
            if first is second:
                continue
            for o in (first, second):
                for n in names:
                    if o.get(n):
                        o[n].t.zero_()
            torch.cuda.synchronize()
            for _ in range(5):
                first["call"]()
                second["call"](side)
            torch.cuda.synchronize()
            for o in (first, second):
                for n, v in want[[o is c for c in cases].index(True)].items():
                    assert torch.equal(o[n].t, v), n
    G.check_no_device_error()


# ---- first calls inside a capture ------------------------------------------------------------------

PROGRAM = r"""
import torch
import nvfp4_precision_transformer_gb300 as te
from nvfp4_precision_transformer_gb300 import _lib as L

BF, U8, ONE = torch.bfloat16, torch.uint8, torch.ones(1, device="cuda")
K, N = 2048, 512
g = torch.Generator(device="cuda").manual_seed(1)


def bytes_(*shape):     # E4M3 codes of moderate size; pairs of E2M1 codes
    return torch.randint(0x28, 0x40, shape, dtype=U8, device="cuda", generator=g)


def mx(r, c):
    return torch.full((L._mx_bytes(r, c),), 118, dtype=U8, device="cuda")


def nv(r, c):
    return torch.full((L._nv_bytes(r, c),), 0x20, dtype=U8, device="cuda")


w16 = torch.randn(N, K, device="cuda", generator=g).mul(0.05).to(BF)
w8, w4 = bytes_(N, K), bytes_(N, K // 2)


def call(kind, T, x, y, db):
    z = torch.ones(T, N, dtype=BF, device="cuda")
    ws = torch.empty(te.te_act_dbias_workspace_bytes(T, max(N, K)) // 4, device="cuda")
    if kind == "bf16":
        te.te_act_gemm_bf16(x, w16, te.ACT_GELU, y=y)
    elif kind == "fp8":
        q = torch.empty(T, N, dtype=U8, device="cuda")
        te.te_act_gemm_fp8(x, te.E4M3, w8, te.E4M3, ONE, ONE, te.ACT_GELU, y=y, q=q, q_scale=ONE, q_amax=db[:1])
    elif kind == "mxfp8":
        te.te_act_gemm_mxfp8(x, mx(T, K), w8, mx(N, K), te.ACT_GELU, y=y)
    elif kind == "nvfp4":
        te.te_act_gemm_nvfp4(x, nv(T, K), ONE, w4, nv(N, K), ONE, te.ACT_GELU, y=y)
    elif kind == "bwd":
        te.te_act_bwd_bf16(x, w16, w16[:, :N].contiguous(), z, z, te.ACT_GELU, y, db, ws, torch.empty_like(x), torch.empty_like(w16))
    elif kind == "dgrad":
        te.te_act_dgrad_fp8(x, te.E4M3, w8, te.E4M3, ONE, ONE, z, te.ACT_GELU, y, db, ws)
    else:
        mu, rs = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
        gamma = torch.ones(K, device="cuda")
        n = torch.empty_like(x)
        te.te_add_layernorm_fp8(x, gamma, gamma, 1e-5, te.E4M3, ONE, torch.empty(T, K, dtype=U8, device="cuda"), y=n, mu=mu,
                                rsigma=rs, amax_out=db[:1])
        te.te_layernorm_bwd(n, x, gamma, mu, rs, torch.empty_like(x), gamma.clone(), gamma.clone(),
                            torch.empty(te.te_layernorm_bwd_workspace_bytes(T, K) // 4, device="cuda"))
        y.copy_(n[:, :N])


def inputs(kind, T):
    if kind in ("bf16", "bwd", "norm"):
        x = torch.randn(T, K, device="cuda", generator=g).to(BF)
    else:
        x = bytes_(T, K if kind != "nvfp4" else K // 2)
    return x, torch.zeros(T, N, dtype=BF, device="cuda"), torch.full((N,), -1.0, device="cuda")


te.te_rmsnorm_fp8(torch.ones(1, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda"), 1e-5, te.E4M3,
                  y=torch.empty(1, 64, dtype=BF, device="cuda"))      # the first call on the device
torch.cuda.synchronize()
for kind in ("bf16", "fp8", "mxfp8", "nvfp4", "bwd", "dgrad", "norm"):
    for T in (1, 20, 40, 100, 300, 2500):
        x, y, db = inputs(kind, T)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(kind, T, x, y, db)
        graph.replay()
        torch.cuda.synchronize()
        got = (y.clone(), db.clone())
        y.zero_()
        db.fill_(-1.0)
        call(kind, T, x, y, db)
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], db), (kind, T)
        assert bool((y != 0).any()), (kind, T)
assert te.te_get_last_error() == 0
print("ok")
"""


def test_first_calls_can_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
