"""The feed-forward block with one activation (norm, up projection, down projection onto the stream) forward and
backward under each recipe, against the 64-bit composition of the oracle's operators.

Tolerances, relative Frobenius, as in test_gpu_gated_mlp: a value that is rounded with half a step r (bf16 2^-8, E4M3
2^-4, E5M2 2^-3, the largest relative error) contributes at most r, and a product of two rounded operands at most the
sum of theirs; the longest chains here round eight operands, five of them to bf16 or E4M3 and three to E5M2.  y, dx
carry the stream beside the block's part and are compared without it (y - s, dx - dy), with the stream's own rounding
on top: 2^-8 of what was rounded."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from nvfp4_precision_transformer_gb300 import _lib as L
from nvfp4_precision_transformer_gb300.mlp import MLP
from oracle.act import act_dgrad, linear_act
from oracle.layernorm import add_layernorm, layernorm_bwd
from tests import gpu_util as G

TOL = {"bf16": 8 * 2.0 ** -8, "fp8_delayed": 5 * 2.0 ** -4 + 3 * 2.0 ** -3, "mxfp8": 8 * 2.0 ** -4}
ACT = {"gelu": te.ACT_GELU, "relu": te.ACT_RELU}


def _case(T, K, F, seed=0):
    g = torch.Generator().manual_seed(seed + T)

    def r(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).bfloat16().to(G.DEV)

    def v(n, mean, std):
        return (mean + std * torch.randn(n, generator=g)).to(G.DEV)

    return (dict(gamma=v(K, 1, 0.1), beta=v(K, 0, 0.1), w1=r(F, K, std=K ** -0.5), b1=v(F, 0, 0.1), w2=r(K, F, std=F ** -0.5),
                 b2=v(K, 0, 0.1)), r(T, K), r(T, K), r(T, K, std=1e-3))


def _off(got, want, base=None):
    """Relative Frobenius error of got - base, less what rounding the sum to bf16 may have left."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    base = 0.0 if base is None else base
    err = np.maximum(np.abs(got - want) - (2.0 ** -8 * np.abs(want) if np.ndim(base) else 0.0), 0.0)
    return np.linalg.norm(err) / np.linalg.norm(want - base)


@pytest.mark.gpu
@pytest.mark.parametrize("recipe", ["bf16", "fp8_delayed", "mxfp8"])
@pytest.mark.parametrize("T,K,F,act,residual", [(64, 256, 384, "gelu", True), (160, 768, 2048, "gelu", False),
                                                (32, 288, 1056, "relu", True)])
def test_block(recipe, T, K, F, act, residual):
    p, x, res, dy = _case(T, K, F)
    res = res if residual else None
    block = MLP(tokens=T, recipe=recipe, act=ACT[act], **p)
    for _ in range(3):                      # fp8_delayed: the scales settle on the history
        y = block.forward(x, res)
        block.backward(dy)
    torch.cuda.synchronize()
    G.check_no_device_error()
    n = {k: v.double().cpu().numpy() for k, v in dict(x=x, dy=dy, **p).items()}
    s64, n64, mu64, rs64 = add_layernorm(n["x"], n["gamma"], n["beta"], block.eps, None if res is None else res.double().cpu().numpy())
    h64, z64, _ = linear_act(n64, n["w1"], act, n["b1"])
    y64, _, _ = linear_act(h64, n["w2"], "none", n["b2"], s64)
    dz64, db1 = act_dgrad(n["dy"], n["w2"], z64, act)
    dx64, dgamma, dbeta = layernorm_bwd(dz64 @ n["w1"], s64, n["gamma"], mu64, rs64, n["dy"])
    tol = TOL[recipe]
    if act == "relu":
        # a z that rounding takes across zero switches its whole gradient: of z's density at zero (below 1 / std), the part
        # within z's own error
        tol += (0.8 * {"bf16": 4 * 2.0 ** -8}.get(recipe, 2 * 2.0 ** -4)) ** 0.5
    assert _off(y, y64, s64) <= tol and _off(block.dx, dx64, n["dy"]) <= tol
    for got, want in ((block.h, h64), (block.dz, dz64), (block.dw2, n["dy"].T @ h64), (block.dw1, dz64.T @ n64),
                      (block.db1, db1), (block.dgamma, dgamma), (block.dbeta, dbeta)):
        assert _off(got, want) <= tol
    # the sum of dy itself: fp32, whatever the recipe
    assert np.all(np.abs(block.db2.cpu().double().numpy() - n["dy"].sum(0)) <= (T + 8) * 2.0 ** -24 * np.abs(n["dy"]).sum(0))


@pytest.mark.gpu
def test_checkpoint_resumes_bit_for_bit():
    p, x, res, dy = _case(64, 256, 384)
    a = MLP(tokens=64, recipe="fp8_delayed", **p)
    for _ in range(2):
        a.forward(x, res)
        a.backward(dy)
    b = MLP(tokens=64, recipe="fp8_delayed", **p)
    b.load_state_dict(a.state_dict())
    for m in (a, b):
        m.forward(x, res)
        m.backward(dy)
    torch.cuda.synchronize()
    for f in ("y", "dx", "dw1", "db1", "dw2", "db2", "dgamma", "dbeta"):
        assert torch.equal(getattr(a, f), getattr(b, f)), f
    assert torch.equal(a.fwd.hist, b.fwd.hist) and torch.equal(a.bwd.scale, b.bwd.scale)


@pytest.mark.gpu
@pytest.mark.parametrize("recipe", ["bf16", "fp8_delayed", "mxfp8"])
def test_a_captured_step(recipe):
    """A step in a graph gives the step's bits (FP8: the scales stay, as the history's slot is the captured one's)."""
    p, x, res, dy = _case(96, 256, 512)
    block = MLP(tokens=96, recipe=recipe, **p)
    block.forward(x, res)
    block.backward(dy)
    names = ("y", "dx", "dw1", "db1", "dw2", "db2", "dgamma", "dbeta")
    graph, step = torch.cuda.CUDAGraph(), block.step_idx
    state = block.state_dict()
    with torch.cuda.graph(graph):
        block.forward(x, res)
        block.backward(dy)
    block.load_state_dict(state)
    graph.replay()
    torch.cuda.synchronize()
    got = [getattr(block, n).clone() for n in names]
    block.load_state_dict(state)
    assert block.step_idx == step
    block.forward(x, res)
    block.backward(dy)
    torch.cuda.synchronize()
    assert all(torch.equal(g, getattr(block, n)) for g, n in zip(got, names))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5])
def test_serving_by_the_calls(T):
    """A few tokens through the same chain without a block: any number of them."""
    p, x, res, _ = _case(T, 768, 2048)
    want = [v.double().cpu().numpy() for v in (x, res)]
    y, h = torch.empty_like(x), torch.empty(T, 2048, dtype=torch.bfloat16, device=G.DEV)
    te.te_add_layernorm_fp8(x, p["gamma"], p["beta"], 1e-5, te.E4M3, residual=res, res_out=res, y=y)
    te.te_act_gemm_bf16(y, p["w1"], te.ACT_GELU, y=h, bias=p["b1"])
    te.te_act_gemm_bf16(h, p["w2"], te.ACT_NONE, y=res, bias=p["b2"], residual=res)
    torch.cuda.synchronize()
    n = {k: v.double().cpu().numpy() for k, v in p.items()}
    s64, n64, _, _ = add_layernorm(want[0], n["gamma"], n["beta"], 1e-5, want[1])
    h64 = linear_act(n64, n["w1"], "gelu", n["b1"])[0]
    # s itself is rounded once more on its way here
    y64 = linear_act(h64, n["w2"], "none", n["b2"], s64)[0]
    err = np.abs(res.double().cpu().numpy() - y64) - 2.0 ** -8 * (np.abs(y64) + np.abs(s64))
    assert np.linalg.norm(np.maximum(err, 0)) <= 6 * 2.0 ** -8 * np.linalg.norm(y64 - s64)


# ---- refusals: nothing reaches the GPU -------------------------------------------------------------

class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def launches(monkeypatch):
    """Names of the launching calls made, none of which reaches the library."""
    made = []
    for name in L.SIGNATURES:
        if hasattr(L, name) and not name.endswith("_bytes") and name not in ("te_status_str", "te_recipe"):
            monkeypatch.setattr(L, name, lambda *a, _n=name, **k: made.append(_n))
    monkeypatch.setattr(L, "_device", lambda: 0)
    return made


F32 = torch.float32
GOOD = dict(gamma=(64, F32), beta=(64, F32), w1=((128, 64), torch.bfloat16), b1=(128, F32), w2=((64, 128), torch.bfloat16), b2=(64, F32))


def params(**other):
    p = {k: gpu(*(s if isinstance(s, tuple) else (s,)), dtype=t) for k, (s, t) in GOOD.items()}
    return {**p, **other}


@pytest.mark.parametrize("recipe", ["bf16", "fp8_delayed", "mxfp8"])
def test_block_refuses_before_it_launches(launches, recipe):
    bad = dict(gamma=gpu(64), beta=gpu(63, dtype=F32), w1=gpu(64, 128).t(), b1=gpu(64, dtype=F32), w2=torch.zeros(64, 128, dtype=torch.bfloat16),
               b2=gpu(64))
    for name, value in bad.items():
        with pytest.raises((TypeError, ValueError)):
            MLP(tokens=32, recipe=recipe, **params(**{name: value}))
        b = MLP(tokens=32, recipe=recipe, **params())
        with pytest.raises(RuntimeError):
            b.backward(gpu(32, 64))
        setattr(b, name, value)
        with pytest.raises((TypeError, ValueError)):
            b.forward(gpu(32, 64))
    for kw in (dict(tokens=33), dict(tokens=0), dict(tokens=32, recipe="nvfp4"), dict(tokens=32, act=9)):
        with pytest.raises(ValueError):
            MLP(**{"recipe": recipe, **params(), **kw})
    b = MLP(tokens=32, recipe=recipe, **params())
    for x in (gpu(16, 64), gpu(32, 64, dtype=F32), gpu(64, 32).t(), torch.zeros(32, 64, dtype=torch.bfloat16)):
        for args in ((x,), (gpu(32, 64), x)):
            with pytest.raises((TypeError, ValueError)):
                b.forward(*args)
    assert launches == []
    b.forward(gpu(32, 64))
    n = len(launches)
    with pytest.raises((TypeError, ValueError)):
        b.backward(gpu(32, 64, dtype=F32))
    assert len(launches) == n and b.step_idx == 0
    b.backward(gpu(32, 64))
    assert len(launches) > n and b.step_idx == 1


def test_fp32_weights_under_the_recipes_that_quantize_them(launches):
    w = dict(w1=gpu(128, 64, dtype=F32), w2=gpu(64, 128, dtype=F32))
    for recipe in ("fp8_delayed", "mxfp8"):
        MLP(tokens=32, recipe=recipe, **params(**w)).forward(gpu(32, 64))
    with pytest.raises(TypeError):
        MLP(tokens=32, **params(**w))
