"""GatedMLP refuses what a launch behind the first one of a pass would refuse: the norm's limits, and tensors off the
16-byte boundaries that the kernels start from.  Runs on the CPU."""
import pytest
import torch

from nvfp4_precision_transformer_gb300.gated import GatedMLP
from tests.test_gated_mlp_arguments import F, F32, K, RECIPES, T, gpu, launches  # noqa: F401
from tests.test_mlp_arguments import off


def weights():
    return dict(gamma=gpu(K, dtype=F32), w=gpu(2 * F, K), w2=gpu(K, F))


@pytest.mark.parametrize("recipe", RECIPES)
def test_the_norms_limits(launches, recipe):  # noqa: F811
    with pytest.raises(ValueError, match="16384"):
        GatedMLP(gpu(16512, dtype=F32), gpu(256, 16512), gpu(16512, 128), T, recipe)
    for eps in (-1e-5, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="eps"):
            GatedMLP(tokens=T, recipe=recipe, eps=eps, **weights())
    assert launches == []


@pytest.mark.parametrize("recipe", RECIPES)
def test_tensors_off_their_boundary(launches, recipe):  # noqa: F811
    for name, t in weights().items():
        bad = off(*t.shape, dtype=t.dtype)
        with pytest.raises(ValueError, match=name):
            GatedMLP(tokens=T, recipe=recipe, **{**weights(), name: bad})
        b = GatedMLP(tokens=T, recipe=recipe, **weights())
        setattr(b, name, bad)
        with pytest.raises(ValueError, match=name):
            b.forward(gpu(T, K), gpu(T, K))
    b = GatedMLP(tokens=T, recipe=recipe, **weights())
    for name, args in (("x", (off(T, K), gpu(T, K))), ("residual", (gpu(T, K), off(T, K)))):
        with pytest.raises(ValueError, match=name):
            b.forward(*args)
    for name, args in (("dout", (off(T, K),)), ("dr", (gpu(T, K), off(T, K)))):
        with pytest.raises(ValueError, match=name):
            b.backward(*args)
    assert launches == [] and b.step_idx == 0
