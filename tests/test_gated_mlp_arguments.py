"""GatedMLP refuses what its kernels would misread -- another shape, dtype or device, a strided
view -- before it launches anything.  Runs on the CPU: tensors that say they are on the GPU, and
the launching calls replaced by a record of their names."""
import pytest
import torch

from nvfp4_precision_transformer_gb300 import _lib as L
from nvfp4_precision_transformer_gb300.gated import GatedMLP

T, K, F = 32, 64, 128
BF, F32 = torch.bfloat16, torch.float32


class OnGpu(torch.Tensor):
    """A CPU tensor that passes for one on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def gpu(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture
def launches(monkeypatch):
    """Names of the launching calls made, none of which reaches the library."""
    made = []
    host = {"te_scale_bytes", "te_rmsnorm_bwd_workspace_bytes", "te_dbias_workspace_bytes", "te_status_str", "te_recipe"}
    for name in L.SIGNATURES:
        if hasattr(L, name) and name not in host:
            monkeypatch.setattr(L, name, lambda *a, _n=name, **k: made.append(_n))
    monkeypatch.setattr(L, "_device", lambda: 0, raising=False)
    return made


def block(recipe="bf16", gamma=None, w=None, w2=None):
    return GatedMLP(gpu(K, dtype=F32) if gamma is None else gamma, gpu(2 * F, K) if w is None else w,
                    gpu(K, F) if w2 is None else w2, T, recipe)


RECIPES = ("bf16", "fp8_delayed", "mxfp8")


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("which", ["more rows", "fewer rows", "more columns", "vector", "strided", "half", "on the CPU"])
def test_backward_refuses_a_gradient(launches, recipe, which):
    bad = {"more rows": gpu(T + 16, K), "fewer rows": gpu(T - 16, K), "more columns": gpu(T, K + 16), "vector": gpu(K),
           "strided": gpu(K, T).t(), "half": gpu(T, K, dtype=torch.float16), "on the CPU": torch.zeros(T, K, dtype=BF)}[which]
    b = block(recipe)
    for args in ((bad,), (gpu(T, K), bad)):          # dout, dr
        with pytest.raises((TypeError, ValueError)):
            b.backward(*args)
        assert launches == [] and b.step_idx == 0


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("which", ["more rows", "strided", "fp32", "on the CPU"])
def test_forward_refuses_an_input(launches, recipe, which):
    bad = {"more rows": gpu(T + 16, K), "strided": gpu(K, T).t(), "fp32": gpu(T, K, dtype=F32),
           "on the CPU": torch.zeros(T, K, dtype=BF)}[which]
    b = block(recipe)
    for args in ((bad, gpu(T, K)), (gpu(T, K), bad)):
        with pytest.raises((TypeError, ValueError)):
            b.forward(*args)
        assert launches == []


@pytest.mark.parametrize("recipe", RECIPES)
@pytest.mark.parametrize("bad", ["strided w", "strided w2", "half w", "half w2", "w2 on the CPU", "gamma in bf16"])
def test_weights(launches, recipe, bad):
    kw = {"strided w": dict(w=gpu(K, 2 * F).t()), "strided w2": dict(w2=gpu(F, K).t()),
          "half w": dict(w=gpu(2 * F, K, dtype=torch.float16)), "half w2": dict(w2=gpu(K, F, dtype=torch.float16)),
          "w2 on the CPU": dict(w2=torch.zeros(K, F, dtype=BF)), "gamma in bf16": dict(gamma=gpu(K))}[bad]
    with pytest.raises((TypeError, ValueError)):
        block(recipe, **kw)
    # a weight that is put in the place of the first one
    b = block(recipe)
    (name, value), = kw.items()
    setattr(b, name, value)
    with pytest.raises((TypeError, ValueError)):
        b.forward(gpu(T, K), gpu(T, K))
    with pytest.raises((TypeError, ValueError)):
        b.backward(gpu(T, K))
    assert launches == []


def test_bf16_takes_bf16_weights_and_gradients(launches):
    for kw in (dict(w=gpu(2 * F, K, dtype=F32)), dict(w2=gpu(K, F, dtype=F32))):
        with pytest.raises(TypeError):
            block("bf16", **kw)
    with pytest.raises(TypeError):
        block("bf16").backward(gpu(T, K, dtype=F32))
    assert launches == []


@pytest.mark.parametrize("recipe", RECIPES)
def test_what_is_right_is_launched(launches, recipe):
    """The quantizers read fp32 as well: fp32 weights and gradients go on working under their recipes."""
    t = BF if recipe == "bf16" else F32
    b = block(recipe, w=gpu(2 * F, K, dtype=t), w2=gpu(K, F, dtype=t))
    b.forward(gpu(T, K), gpu(T, K))
    b.forward(gpu(T, K), None)
    b.backward(gpu(T, K, dtype=t), gpu(T, K))
    b.backward(gpu(T, K))
    assert len(launches) >= 10 and b.step_idx == 2
