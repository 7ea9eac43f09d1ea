"""The gated feed-forward block (norm, gated projections, down projection) forward and backward
under each recipe, against the 64-bit composition of the oracle's operators.

Tolerances, relative Frobenius: a value that is rounded with half a step r (bf16 2^-8, E4M3 2^-4,
E5M2 2^-3, the largest relative error) contributes at most r, and a product of two rounded operands
at most the sum of theirs; the longest chains here round eight operands (dw in FP8: y, w, h's gates,
dout, w2, dgu, the output), five of them to bf16 or E4M3 and three to E5M2."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from nvfp4_precision_transformer_gb300.gated import GatedMLP
from oracle.gated import gated, gated_bwd
from oracle.rmsnorm import rmsnorm, rmsnorm_bwd
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

TOL = {"bf16": 8 * 2.0 ** -8, "fp8_delayed": 5 * 2.0 ** -4 + 3 * 2.0 ** -3, "mxfp8": 8 * 2.0 ** -4}


def _case(T, K, F, seed=0):
    g = torch.Generator().manual_seed(seed + T)

    def r(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).bfloat16().to(G.DEV)

    gamma = (1 + 0.1 * torch.randn(K, generator=g)).to(G.DEV)
    return gamma, r(2 * F, K, std=K ** -0.5), r(K, F, std=F ** -0.5), r(T, K), r(T, K), r(T, K, std=1e-3), r(T, K, std=1e-3)


def _rel(a, b):
    a = a.double().cpu().numpy()
    assert np.isfinite(a).all()
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("recipe", ["bf16", "fp8_delayed", "mxfp8"])
@pytest.mark.parametrize("T,K,F", [(64, 256, 384), (160, 768, 2048)])
def test_block(recipe, T, K, F):
    gamma, w, w2, x, res, dout, dr = _case(T, K, F)
    block = GatedMLP(gamma, w, w2, T, recipe)
    for _ in range(3):                      # fp8_delayed: the scales settle on the history
        out, r = block.forward(x, res)
        block.backward(dout, dr)
    torch.cuda.synchronize()
    G.check_no_device_error()
    n = {k: v.double().cpu().numpy() for k, v in dict(gamma=gamma, w=w, w2=w2, x=x, res=res, dout=dout, dr=dr).items()}
    s64, y64, rs64 = rmsnorm(n["x"], n["gamma"], block.eps, n["res"])
    h64, g64, u64 = gated(y64, n["w"], "silu")
    dgu = np.concatenate(gated_bwd(n["dout"], n["w2"], g64, u64, "silu"), 1)
    dx64, dgamma64 = rmsnorm_bwd(dgu @ n["w"], s64, n["gamma"], rs64, n["dr"])
    tol = TOL[recipe]
    assert _rel(r, s64) <= 2.0 ** -8
    for got, want in ((out, h64 @ n["w2"].T), (block.h, h64), (block.dgu, dgu), (block.dw2, n["dout"].T @ h64),
                      (block.dw, dgu.T @ y64), (block.dx, dx64), (block.dgamma, dgamma64)):
        assert _rel(got, want) <= tol


def test_checkpoint_resumes_bit_for_bit():
    gamma, w, w2, x, res, dout, dr = _case(64, 256, 384)
    a = GatedMLP(gamma, w, w2, 64, "fp8_delayed")
    for _ in range(2):
        a.forward(x, res)
        a.backward(dout, dr)
    b = GatedMLP(gamma, w, w2, 64, "fp8_delayed")
    b.load_state_dict(a.state_dict())
    for m in (a, b):
        m.forward(x, res)
        m.backward(dout, dr)
    torch.cuda.synchronize()
    for f in ("out", "dx", "dw", "dw2", "dgamma"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    assert torch.equal(a.fwd.hist, b.fwd.hist) and torch.equal(a.bwd.scale, b.bwd.scale)


def test_any_token_count_in_bf16_decode():
    """One token through the norm and the gated projections (the serving form)."""
    gamma, w, w2, x, res, _, _ = _case(1, 768, 2048)
    y, h = torch.empty_like(x), torch.empty(1, 2048, dtype=torch.bfloat16, device=G.DEV)
    te.te_rmsnorm_fp8(x, gamma, 1e-5, te.E4M3, residual=res, res_out=res, y=y)
    te.te_gated_gemm_bf16(y, w, te.ACT_GELU, h=h)
    torch.cuda.synchronize()
    gamma, w, w2, x, res, _, _ = _case(1, 768, 2048)
    _, y64, _ = rmsnorm(x.double().cpu().numpy(), gamma.double().cpu().numpy(), 1e-5, res.double().cpu().numpy())
    h64, _, _ = gated(y64, w.double().cpu().numpy(), "gelu")
    assert _rel(h, h64) <= 4 * 2.0 ** -8


def test_refusals():
    gamma, w, w2, *_ = _case(16, 64, 128)
    with pytest.raises(ValueError):
        GatedMLP(gamma, w, w2, 16, "nvfp4")
    with pytest.raises(ValueError):
        GatedMLP(gamma, w, w2.t().contiguous(), 16)
