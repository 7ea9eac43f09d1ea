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
from tests.test_gpu_act_forms import form

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


def _codes(t, kind):
    return t.bfloat16() if kind == "bf16" else t.to(torch.float8_e4m3fn).view(torch.uint8)


def operands(kind, T, K, N):
    """x and w on the GPU, their product in 64 bits, and the products' factors of the rows and columns."""
    rows = torch.exp2(-torch.arange(T, device=G.DEV).remainder(3).float())
    cols = torch.exp2(-torch.arange(N, device=G.DEV).remainder(2).float())
    x = _codes(rows[:, None] * (1.0 if kind == "bf16" else 16.0), kind).expand(T, K).contiguous()
    w = _codes(cols[:, None] * _pattern(kind).to(G.DEV)[None, :], kind).repeat(1, K // TERMS[kind])
    return x, w, float(GROUP[kind]) * (K // TERMS[kind]) * (rows.double()[:, None] * cols.double()[None, :])


def scales(R, C):
    return torch.full((te.te_scale_bytes(te.E8M0, R, C),), 127, dtype=torch.uint8, device=G.DEV)


def segments(kind, K):
    """Segments of a contraction, and of one whose parts (eight at most) have a shorter last one each."""
    return -(-K // SEGMENT[kind]) + 8


def lost_in_one_piece(kind, n):
    """What n groups lose of their 15 where each addition rounds towards zero."""
    total = exact = 0
    for _ in range(n):
        exact += GROUP[kind]
        total += GROUP[kind]
        total -= total % max(1, 2 ** (total.bit_length() - 24))
    return exact - total


def allowed(kind, K, want):
    return segments(kind, K) * 2.0 ** -24 * want.abs()


FORMS = [("bf16", 1, 65536, 4112, "stream shared"), ("bf16", 24, 16384, 20016, "stream"), ("bf16", 2080, 65536, 272, "pair shared"),
         ("bf16", 2080, 16384, 3344, "pair"), ("fp8", 24, 131072, 10256, "stream"), ("fp8", 2080, 131072, 272, "pair shared"),
         ("fp8", 2080, 131072, 3344, "pair"), ("mxfp8", 24, 131072, 10256, "stream"), ("mxfp8", 2080, 131072, 272, "pair"),
         ("mxfp8", 2080, 131072, 3360, "pair")]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,K,N,what", FORMS)
def test_forward(kind, T, K, N, what):
    x, w, want = operands(kind, T, K, N)
    y = torch.zeros(T, N, device=G.DEV)
    one = G.scalar(1.0)

    def call(stream=None):
        if kind == "bf16":
            te.te_act_gemm_bf16(x, w, te.ACT_NONE, y=y, stream=stream)
        elif kind == "fp8":
            te.te_act_gemm_fp8(x, te.E4M3, w, te.E4M3, one, one, te.ACT_NONE, y=y, stream=stream)
        else:
            te.te_act_gemm_mxfp8(x, sx, w, sw, te.ACT_NONE, y=y, stream=stream)

    sx, sw = (scales(T, K), scales(N, K)) if kind == "mxfp8" else (None, None)
    call()
    torch.cuda.synchronize()
    G.check_no_device_error()
    assert bool(((y.double() - want).abs() <= allowed(kind, K, want)).all()), float((y.double() / want - 1).abs().max())
    assert form(call)[0] == what


# dh of one token is dbias itself; few columns (a tile shared by pairs, where the kind has that form) and more tiles than pairs
@pytest.mark.gpu
@pytest.mark.parametrize("kind,N,F", [("bf16", 65536, 272), ("bf16", 16384, 20016), ("fp8", 131072, 272), ("fp8", 131072, 20016),
                                      ("mxfp8", 131072, 272), ("mxfp8", 131072, 20032)])
def test_dgrad(kind, N, F):
    d, w, want = operands(kind, 1, N, F)
    dz, db = torch.zeros(1, F, dtype=torch.bfloat16, device=G.DEV), torch.zeros(F, device=G.DEV)
    ws = torch.empty(te.te_act_dbias_workspace_bytes(1, F) // 4, device=G.DEV)
    one = G.scalar(1.0)
    sd, sw = (scales(1, N), scales(F, N)) if kind == "mxfp8" else (None, None)
    w2 = w.t().contiguous() if kind == "bf16" else w

    def call(stream=None):
        kw = dict(dbias=db, workspace=ws, stream=stream)
        if kind == "bf16":
            te.te_act_bwd_bf16(torch.zeros(1, 16, dtype=torch.bfloat16, device=G.DEV),
                               torch.zeros(F, 16, dtype=torch.bfloat16, device=G.DEV), w2, d, None, te.ACT_NONE, dz, **kw)
        elif kind == "fp8":
            te.te_act_dgrad_fp8(d, te.E4M3, w2, te.E4M3, one, one, None, te.ACT_NONE, dz, **kw)
        else:
            te.te_act_dgrad_mxfp8(d, sd, w2, sw, None, te.ACT_NONE, dz, **kw)

    call()
    torch.cuda.synchronize()
    G.check_no_device_error()
    assert bool(((db.double() - want[0]).abs() <= allowed(kind, N, want[0])).all()), float((db.double() / want[0] - 1).abs().max())
    assert form(call)[0] == ("pair shared" if F == 272 and kind != "mxfp8" else "pair")


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


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,what", [(24, 10256, "stream"), (2080, 272, "pair shared"), (2080, 3344, "pair")])
def test_amax_of_the_8_bit_output(T, N, what):
    """An fp32 output too, whether y is there or not."""
    K = 131072
    x, w, want = operands("fp8", T, K, N)
    q, y, amax, one = G.u8(T, N), torch.zeros(T, N, dtype=torch.bfloat16, device=G.DEV), G.scalar(-1.0), G.scalar(1.0)
    for kw in (dict(), dict(y=y)):
        def call(stream=None):
            te.te_act_gemm_fp8(x, te.E4M3, w, te.E4M3, one, one, te.ACT_NONE, q=q, q_scale=one, q_amax=amax, stream=stream, **kw)

        call()
        torch.cuda.synchronize()
        G.check_no_device_error()
        top = want.max()
        assert bool((amax.double() - top).abs() <= allowed("fp8", K, top)), amax.item() / top.item() - 1
        assert form(call)[0] == what


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp8", "mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,K,N", [(24, 32768, 4096), (300, 32768, 1056), (2080, 16512, 3360)])
def test_outputs_do_not_depend_on_one_another(kind, T, K, N):
    """z and q, bit for bit, with y in bf16, in fp32 and without it."""
    g = torch.Generator(device=G.DEV).manual_seed(T)
    codes = lambda *shape: torch.randint(0x20, 0x40, shape, dtype=torch.uint8, device=G.DEV, generator=g) + (   # noqa: E731
        torch.randint(0, 2, shape, dtype=torch.uint8, device=G.DEV, generator=g) * 128)
    x, w = (codes(T, K), codes(N, K)) if kind != "nvfp4" else (codes(T, K // 2), codes(N, K // 2))
    bias, one = torch.randn(N, device=G.DEV, generator=g), G.scalar(1.0)
    if kind == "nvfp4":
        sx, sw = (torch.full((te.te_scale_bytes(te.UE4M3, r, K),), 0x28, dtype=torch.uint8, device=G.DEV) for r in (T, N))
    else:
        sx, sw = scales(T, K), scales(N, K).fill_(118)
    first = {}
    for yt in (None, torch.bfloat16, torch.float32):
        out = dict(z=torch.zeros(T, N, dtype=torch.bfloat16, device=G.DEV))
        more = dict(y=None if yt is None else torch.zeros(T, N, dtype=yt, device=G.DEV), z=out["z"], bias=bias)
        if kind != "nvfp4":
            out["q"] = more["q"] = G.u8(T, N)
        if kind == "fp8":
            out["amax"] = more["q_amax"] = G.scalar(-1.0)
            te.te_act_gemm_fp8(x, te.E4M3, w, te.E4M3, one, G.scalar(2.0 ** -9), te.ACT_GELU, q_scale=one, **more)
        elif kind == "mxfp8":
            out["s"] = more["s_q"] = torch.zeros(te.te_scale_bytes(te.E8M0, T, N), dtype=torch.uint8, device=G.DEV)
            te.te_act_gemm_mxfp8(x, sx, w, sw, te.ACT_GELU, **more)
        else:
            te.te_act_gemm_nvfp4(x, sx, one, w, sw, one, te.ACT_GELU, **more)
        torch.cuda.synchronize()
        G.check_no_device_error()
        for n, v in out.items():
            assert torch.equal(first.setdefault(n, v), v), (yt, n)
    assert bool((first["z"].float().abs() > 0.01).float().mean() > 0.9) and bool(first["z"].isfinite().all())


def test_what_one_piece_would_lose():
    """The cases tell a cut sum from an uncut one: also where eight, four or two CTAs or pairs have a part each."""
    for kind, K, parts in (("bf16", 16384, 1), ("bf16", 65536, 4), ("bf16", 65536, 8), ("fp8", 131072, 4), ("mxfp8", 131072, 1)):
        n = K // TERMS[kind]
        assert parts * lost_in_one_piece(kind, n // parts) > 3 * segments(kind, K) * 2.0 ** -24 * GROUP[kind] * n, (kind, K)
