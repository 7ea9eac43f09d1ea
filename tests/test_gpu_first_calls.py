"""First calls of a form of the gated kernels, with the look-ups that they make, inside a stream capture, after
one call of another form: the graph gives the bits of the call made on its own."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import torch
import nvfp4_precision_transformer_gb300 as te
from nvfp4_precision_transformer_gb300 import _lib as L

BF, U8, ONE = torch.bfloat16, torch.uint8, torch.ones(1, device="cuda")
K, F = 2048, 512
g = torch.Generator(device="cuda").manual_seed(1)


def bytes_(*shape):     # E4M3 codes of moderate size; pairs of E2M1 codes
    return torch.randint(0x28, 0x40, shape, dtype=U8, device="cuda", generator=g)


w16 = torch.randn(2 * F, K, device="cuda", generator=g).mul(0.05).to(BF)
w8, w4 = bytes_(2 * F, K), bytes_(2 * F, K // 2)
mx = torch.full((L._mx_bytes(2 * F, K),), 118, dtype=U8, device="cuda")
nv = torch.full((L._nv_bytes(2 * F, K),), 0x20, dtype=U8, device="cuda")


def call(kind, T, x, h, amax):
    if kind == "bf16":
        te.te_gated_gemm_bf16(x, w16, te.ACT_SILU, h=h)
    elif kind == "fp8":
        q = torch.empty(T, F, dtype=U8, device="cuda")
        te.te_gated_gemm_fp8(x, te.E4M3, w8, te.E4M3, ONE, ONE, te.ACT_SILU, h=h, q_h=q, h_scale=ONE, h_amax=amax)
    elif kind == "mxfp8":
        te.te_gated_gemm_mxfp8(x, mx, w8, mx, te.ACT_SILU, h=h)
    elif kind == "nvfp4":
        te.te_gated_gemm_nvfp4(x, nv, ONE, w4, nv, ONE, te.ACT_SILU, h=h)
    else:
        gu = torch.ones(T, 2 * F, dtype=BF, device="cuda")
        te.te_gated_bwd_bf16(x, w16, w16[:F, :F].contiguous(), h, gu, te.ACT_SILU, torch.empty_like(gu),
                             dx=torch.empty_like(x), dw=torch.empty_like(w16))


def inputs(kind, T):
    if kind in ("bf16", "bwd"):
        x = torch.randn(T, K, device="cuda", generator=g).to(BF)
    else:
        x = bytes_(T, K if kind != "nvfp4" else K // 2)
    return x, torch.zeros(T, F, dtype=BF, device="cuda"), torch.full((1,), -1.0, device="cuda")


call("bf16", 24, *inputs("bf16", 24))          # the first call on the device
torch.cuda.synchronize()
for kind in ("bf16", "fp8", "mxfp8", "nvfp4", "bwd"):
    for T in (1, 20, 24, 40, 100, 300):
        x, h, amax = inputs(kind, T)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(kind, T, x, h, amax)
        graph.replay()
        torch.cuda.synchronize()
        got = (h.clone(), amax.clone())
        h.zero_()
        amax.fill_(-1.0)
        call(kind, T, x, h, amax)
        torch.cuda.synchronize()
        assert torch.equal(got[0], h) and torch.equal(got[1], amax), (kind, T)
        assert kind == "bwd" or bool((h != 0).any()), (kind, T)
assert te.te_get_last_error() == 0
print("ok")
"""


@pytest.mark.gpu
def test_first_calls_can_be_captured():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
