"""te_act_bwd_bf16 asks for x where dW is wanted and for w where dX is, and for neither where dz alone is."""
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G
from tests.test_wrapper_devices import F32, gpu, library  # noqa: F401

T, K, F, N = 32, 64, 128, 48


def base():
    return dict(w2=gpu(N, F), dy=gpu(T, N), z=gpu(T, F), act=te.ACT_GELU, dz=gpu(T, F), stream=7)


@pytest.mark.parametrize("wanted", [(), ("dx",), ("dw",), ("dx", "dw")])
def test_what_is_not_read_is_not_asked_for(library, wanted):  # noqa: F811
    out = {n: gpu(T, K) if n == "dx" else gpu(F, K, dtype=F32) for n in wanted}
    ops = dict(x=gpu(T, K) if "dw" in wanted else None, w=gpu(F, K) if "dx" in wanted else None)
    te.te_act_bwd_bf16(**ops, **out, **base())
    assert library.calls == ["te_act_bwd_bf16"]
    for name, value in ops.items():
        if value is not None:
            with pytest.raises(TypeError, match=name):
                te.te_act_bwd_bf16(**{**ops, name: None}, **out, **base())
    assert len(library.calls) == 1


def test_shapes_that_do_not_fit_are_refused(library):  # noqa: F811
    good = dict(base(), x=gpu(T, K), w=gpu(F, K), dx=gpu(T, K), dw=gpu(F, K))
    bad = dict(x=(gpu(T, K + 16), gpu(T + 16, K), gpu(K)), w=(gpu(F, K + 16), gpu(F + 16, K), gpu(K)), w2=(gpu(N + 16, F), gpu(F)),
               dy=(gpu(T, N + 16), gpu(N)), dx=(gpu(T, K + 16),), dw=(gpu(K, F),), z=(gpu(T, F + 16),), dz=(gpu(T + 16, F),))
    for name, values in bad.items():
        for v in values:
            with pytest.raises(ValueError):
                te.te_act_bwd_bf16(**{**good, name: v})
    assert library.calls == []


@pytest.mark.gpu
def test_the_same_dz_and_gradients_without_what_is_not_read():
    g = torch.Generator(device=G.DEV).manual_seed(5)
    r = lambda *s: torch.randn(*s, device=G.DEV, generator=g).bfloat16()   # noqa: E731
    x, w, w2, dy, z = r(T, K), r(F, K), r(N, F), r(T, N), r(T, F)
    ws = torch.empty(te.te_act_dbias_workspace_bytes(T, F) // 4, device=G.DEV)
    new = lambda: (torch.zeros_like(z), torch.zeros(F, device=G.DEV), torch.zeros_like(x), torch.zeros_like(w))   # noqa: E731
    dz, db, dx, dw = new()
    te.te_act_bwd_bf16(x, w, w2, dy, z, te.ACT_GELU, dz, db, ws, dx, dw)
    for take in ((), ("dx",), ("dw",)):
        dz2, db2, dx2, dw2 = new()
        te.te_act_bwd_bf16(x if "dw" in take else None, w if "dx" in take else None, w2, dy, z, te.ACT_GELU, dz2, db2, ws,
                           dx2 if "dx" in take else None, dw2 if "dw" in take else None)
        torch.cuda.synchronize()
        assert torch.equal(dz, dz2) and torch.equal(db, db2)
        assert torch.equal(dx2, dx if "dx" in take else torch.zeros_like(dx))
        assert torch.equal(dw2, dw if "dw" in take else torch.zeros_like(dw))
    assert bool(dx.any()) and bool(dw.any())
    G.check_no_device_error()
