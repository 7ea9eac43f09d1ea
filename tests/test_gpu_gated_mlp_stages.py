"""GatedMLP on the GPU, stage by stage from the tensors that each kernel read (gated_stages.verify)."""
import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from nvfp4_precision_transformer_gb300.gated import GatedMLP
from tests import gpu_util as G
from tests.gated_stages import verify
from tests.test_gpu_gated_mlp import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("recipe", ["bf16", "fp8_delayed", "mxfp8"])
@pytest.mark.parametrize("T,K,F", [(64, 256, 384), (160, 768, 2048), (32, 512, 1024)])
def test_stages(recipe, T, K, F):
    gamma, w, w2, x, res, dout, dr = _case(T, K, F, 9)
    block = GatedMLP(gamma, w, w2, T, recipe)
    scale = {}
    for _ in range(3):                       # the FP8 scales settle on the history
        if recipe == "fp8_delayed":          # those of this step: the end of the backward pass moves them on
            scale = {n: (s[0].clone(), s[1].clone()) for n, s in block.slots.items()}
        block.forward(x, res)
        block.backward(dout, dr)
    torch.cuda.synchronize()
    G.check_no_device_error()
    t = dict(gamma=gamma, w=w, w2=w2, x=x, res=res, dout=dout, dr=dr)
    t.update({n: getattr(block, n) for n in ("r", "y", "rsigma", "gu", "h", "out", "dgu", "dy", "dx", "dw", "dw2", "dgamma")})
    t = {n: v.detach().cpu().double().numpy() for n, v in t.items()}
    if recipe != "bf16":
        t["row"] = {n: v.cpu().numpy() for n, v in block.row.items()}
        t["col"] = {n: v.cpu().numpy() for n, v in block.col.items()}
    if recipe == "mxfp8":
        for key, copies, codes in (("srow", block.srow, block.row), ("scol", block.scol, block.col)):
            t[key] = {n: te.te_scale_unswizzle(te.E8M0, *codes[n].shape, v.cpu().numpy()) for n, v in copies.items()}
    if recipe == "fp8_delayed":
        t["scale"], t["inv"] = ({n: np.float32(s[i].item()) for n, s in scale.items()} for i in (0, 1))
        # each tensor's amax went to its own slot
        for n in ("w", "w2", "dout", "dgu"):
            assert block.slots[n][2].item() == np.abs(t[n]).max(), n
        for n in ("y", "h"):
            top = np.abs(t[n]).max()
            assert abs(block.slots[n][2].item() - top) <= 2.0 ** -8 * top, n
    verify(t, recipe)
