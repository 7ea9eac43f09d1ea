"""Long sums in fp32: a contraction is cut into segments, and their sums are added rounding to nearest, in every kernel
that has an fp32 output.

The tensor cores round each addition to an accumulator towards zero.  Each group of terms (what one instruction
multiplies, 16 in BF16 and 32 in 8 bits) adds 2^k + 15 here, so that a segment's sum is a whole number below 2^24, held
exactly, and the whole sum is 2^26 to 2^28 and more: in one piece every group past 2^24 would lose a part of its 15,
together more than three times what is allowed: half a step of fp32, 2^-24 of the sum at most, for each addition of a
segment or of a part of the contraction.  Rows and columns differ by powers of two, which change no rounding."""
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G

SEGMENT = {"bf16": 13 * 64, "fp8": 64 * 128, "mxfp8": 64 * 128}      # elements
GROUP = {"bf16": 2 ** 18 + 15, "fp8": 2 ** 15 + 15, "mxfp8": 2 ** 15 + 15}
TERMS = {"bf16": 16, "fp8": 32, "mxfp8": 32}


def _pattern(kind):
    """A group's terms: the weights' values, beside operands of 1 (BF16) and 16 (8 bits)."""
    v = torch.zeros(TERMS[kind])
    if kind == "bf16":
        v[3], v[9] = 2.0 ** 18, 15.0
    else:
        v[1:30:4] = 256.0                                       # 8 x 256 x 16
        v[30] = 0.9375
    return v


def segments(kind, K):
    """Segments of a contraction, and of one whose parts (eight at most) have a shorter last one each."""
    return -(-K // SEGMENT[kind]) + 8


def allowed(kind, K, want):
    return segments(kind, K) * 2.0 ** -24 * want.abs()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,F", [(65536, 16, 272), (16384, 2064, 2576), (65539, 208, 272)])
def test_weight_gradient_in_fp32(T, K, F):
    """dW of te_act_bwd_bf16 is a sum over the tokens: dz is 2^18, 15 and zeros, x ones.  Alone, beside dX, and added to
    what dW holds."""
    n = T // 16
    t = torch.arange(T, device=G.DEV)
    row = torch.where(t < 16 * n, _pattern("bf16").to(G.DEV)[t % 16], 0.0)
    dy = torch.zeros(T, 16, dtype=torch.bfloat16, device=G.DEV)
    dy[:, 5] = row.bfloat16()
    rows = torch.exp2(-torch.arange(F, device=G.DEV).remainder(3).float())
    cols = torch.exp2(-torch.arange(K, device=G.DEV).remainder(2).float())
    w2 = torch.zeros(16, F, dtype=torch.bfloat16, device=G.DEV)
    w2[5] = rows.bfloat16()
    x = cols.bfloat16().expand(T, K).contiguous()
    w = torch.zeros(F, K, dtype=torch.bfloat16, device=G.DEV)
    want = float(GROUP["bf16"]) * n * (rows.double()[:, None] * cols.double()[None, :])
    dz, dx, dw = torch.zeros(T, F, dtype=torch.bfloat16, device=G.DEV), torch.zeros_like(x), torch.zeros(F, K, device=G.DEV)
    for kw in (dict(), dict(dx=dx), dict(accumulate=1), dict(dx=dx, accumulate=1)):
        before = torch.full_like(dw, 2.0 ** 20)
        dw.copy_(before)
        te.te_act_bwd_bf16(x, w, w2, dy, None, te.ACT_NONE, dz, dw=dw, **kw)
        torch.cuda.synchronize()
        G.check_no_device_error()
        total = want + before.double() if "accumulate" in kw else want
        assert bool(((dw.double() - total).abs() <= allowed("bf16", T, total)).all()), (kw, float((dw.double() / total - 1).abs().max()))
