"""MLP refuses what a launch behind the first one of a pass would refuse: the norm's limits, and tensors off the 16-byte
boundaries that the kernels start from.  Runs on the CPU."""
import pytest
import torch

from nvfp4_precision_transformer_gb300.mlp import MLP
from tests.test_gpu_mlp import GOOD, gpu, launches, params  # noqa: F401

RECIPES = ("bf16", "fp8_delayed", "mxfp8")


@pytest.mark.parametrize("recipe", RECIPES)
def test_the_norms_limits(launches, recipe):  # noqa: F811
    wide = dict(gamma=gpu(16416, dtype=torch.float32), beta=gpu(16416, dtype=torch.float32), w1=gpu(32, 16416),
                b1=gpu(32, dtype=torch.float32), w2=gpu(16416, 32), b2=gpu(16416, dtype=torch.float32))
    with pytest.raises(ValueError, match="16384"):
        MLP(tokens=32, recipe=recipe, **wide)
    for eps in (-1e-5, float("nan"), float("inf"), -float("inf"), 1e39):
        with pytest.raises(ValueError, match="eps"):
            MLP(tokens=32, recipe=recipe, eps=eps, **params())
    assert launches == []
    MLP(tokens=32, recipe=recipe, eps=0.0, **params()).forward(gpu(32, 64))
    assert launches


def off(*shape, dtype=torch.bfloat16):
    """A contiguous view that starts two or four bytes behind a boundary."""
    n = 1
    for k in shape:
        n *= k
    return gpu(n + 1, dtype=dtype)[1:].view(*shape)


@pytest.mark.parametrize("recipe", RECIPES)
def test_tensors_off_their_boundary(launches, recipe):  # noqa: F811
    for name, (shape, dtype) in GOOD.items():
        bad = off(*(shape if isinstance(shape, tuple) else (shape,)), dtype=dtype)
        with pytest.raises(ValueError, match=name):
            MLP(tokens=32, recipe=recipe, **params(**{name: bad}))
        b = MLP(tokens=32, recipe=recipe, **params())
        setattr(b, name, bad)
        with pytest.raises(ValueError, match=name):
            b.forward(gpu(32, 64))
    b = MLP(tokens=32, recipe=recipe, **params())
    for name, args in (("x", (off(32, 64),)), ("residual", (gpu(32, 64), off(32, 64)))):
        with pytest.raises(ValueError, match=name):
            b.forward(*args)
    assert launches == []
    b.forward(gpu(32, 64))
    n = len(launches)
    with pytest.raises(ValueError, match="dy"):
        b.backward(off(32, 64))
    assert len(launches) == n and b.step_idx == 0


@pytest.mark.parametrize("recipe", RECIPES)
def test_the_quantizers_limit(launches, monkeypatch, recipe):  # noqa: F811
    """2^34 elements of dy or, where it is quantized, of h."""
    wide = dict(w1=gpu(1 << 14, 64), b1=gpu(1 << 14, dtype=torch.float32), w2=gpu(64, 1 << 14))
    cases = [dict(tokens=1 << 28, **params())]
    if recipe != "bf16":
        cases.append(dict(tokens=1 << 20, **params(**wide)))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocates before it refuses"))
    for kw in cases:
        with pytest.raises(ValueError, match="quantizer"):
            MLP(recipe=recipe, **kw)
    assert launches == []
