"""The norm and the gated projections of a transformer layer: measured cases and their plain forms.

Four passes of the pre-norm gated feed-forward half of a layer, each in the quantized formats of
this package (FP8 with one scale a tensor, MXFP8, NVFP4) or in BF16:

  norm       r = x + residual;  y = r / sqrt(mean(r^2) + eps) * gamma, and y in 8 bits with scales
  norm_bwd   the gradients of x (and of the residual, the same tensor) and of gamma
  gated      h = act(x Wg^T) * (x Wu^T), Wg and Wu the halves of w [2 F, K]; h in BF16 or in 8 bits,
             and g, u = x w^T where the backward pass keeps them
  gated_bwd  from the gradient dy of y = h w2^T: the gradients of g and u, and (BF16) of x and w

`run` computes them in elementary torch operations, or (`own`) with the package's calls.
8-bit outputs are float8 tensors (views of the bytes), their scales beside them.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -------------------------------------------------------------------------------------
# tokens 15872 = 31 x 512, hidden 4096, intermediate 16384: the CodonFM-5B layer of the benchmark;
# 768 and 1024: the FP8 tutorial's linear.

def listed():
    return [
        # decoding one token with the FP8 recipe: the norm before the feed-forward block
        dict(name="norm_fp8_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, out="fp8", fmt="e4m3",
             keep=False),
        # a tutorial-sized model in training with an odd number of rows and an fp32 residual stream
        dict(name="norm_fp8_fp32_odd", op="norm", rows=1023, cols=768, dtype="fp32", residual=True, out="fp8",
             fmt="e4m3", keep=True),
        # the norm of a training layer under MXFP8: everything that its backward pass needs is kept
        dict(name="norm_mxfp8_layer", op="norm", rows=15872, cols=4096, dtype="bf16", residual=True, out="mxfp8",
             fmt="e4m3", keep=True),
        # its backward pass, with the gradient that comes down the residual stream
        dict(name="norm_bwd_layer", op="norm_bwd", rows=15872, cols=4096, dtype="bf16", residual=True),
        # decoding one token: both weight halves are read for one row
        dict(name="gated_bf16_token", op="gated", kind="bf16", T=1, K=4096, F=16384, act="silu", out="bf16", keep=False),
        # a batch of requests that decode together, FP8 weights
        dict(name="gated_fp8_batch", op="gated", kind="fp8", T=24, K=4096, F=16384, act="silu", out="fp8", keep=False),
        # one sequence of training or prefill, a ragged token count, pre-activations kept
        dict(name="gated_bf16_sequence", op="gated", kind="bf16", T=509, K=4096, F=16384, act="gelu", out="bf16",
             keep=True),
        # the training layer under FP8: h leaves in FP8 for the down projection
        dict(name="gated_fp8_layer", op="gated", kind="fp8", T=15872, K=4096, F=16384, act="silu", out="fp8", keep=True),
        # prefill of eight sequences under MXFP8
        dict(name="gated_mxfp8_prefill", op="gated", kind="mxfp8", T=4096, K=4096, F=16384, act="silu", out="mxfp8",
             keep=False),
        # the training layer under NVFP4
        dict(name="gated_nvfp4_layer", op="gated", kind="nvfp4", T=15872, K=4096, F=16384, act="silu", out="bf16",
             keep=True),
        # a tutorial-sized backward pass with a ragged token count
        dict(name="gated_bwd_bf16_odd", op="gated_bwd", kind="bf16", T=1001, K=768, F=2048, N=768, act="gelu"),
        # the training layer's backward pass: the largest case
        dict(name="gated_bwd_bf16_layer", op="gated_bwd", kind="bf16", T=15872, K=4096, F=16384, N=4096, act="silu"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _mult(rng, lo, hi, m):
    return max(1, round(_log(rng, lo, hi) / m)) * m


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_bwd", "gated", "gated", "gated", "gated_bwd", "gated_bwd"))
    if op in ("norm", "norm_bwd"):
        out = rng.choice(("fp8", "mxfp8"))
        cols = _mult(rng, 64, 16384, 32 if out == "mxfp8" and op == "norm" else 16)
        rows = min(int(_log(rng, 1, 16384)), 15872 * 4096 // cols)
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(("bf16", "fp32")), residual=rng.random() < 0.75)
        if op == "norm":
            case.update(out=out, fmt=rng.choice(("e4m3", "e5m2")) if out == "fp8" else "e4m3", keep=rng.random() < 0.5)
        return case
    kind = rng.choice(("bf16", "fp8", "mxfp8", "nvfp4"))
    block = kind in ("mxfp8", "nvfp4")
    T = int(_log(rng, 1, 15872))
    K = _mult(rng, 64, 8192, 32 if block else 16)
    F = _mult(rng, 128, 16384, 128 if block else 16)
    while T * K * F > 15872 * 4096 * 16384:
        T //= 2
    case = dict(op=op, kind=kind, T=T, K=K, F=F, act=rng.choice(("silu", "gelu")))
    if op == "gated":
        case.update(out=rng.choice(("bf16", kind)) if kind in ("fp8", "mxfp8") else "bf16", keep=rng.random() < 0.5)
    else:
        case.update(N=K)
    return case


def work(case):
    if case["op"] in ("norm", "norm_bwd"):
        n, e = case["rows"] * case["cols"], 4 if case["dtype"] == "fp32" else 2
        r = 1 if case["residual"] else 0
        if case["op"] == "norm":
            b = n * (e + 2 * e * r + 1 + (2 if case["keep"] else 0)) + (n // 32 if case["out"] == "mxfp8" else 0)
            return {"bytes": b + 4 * case["cols"], "flops": 6 * n}
        return {"bytes": n * (2 + 2 * e + e * r) + 8 * case["cols"] + 4 * case["rows"], "flops": 12 * n}
    T, K, F = case["T"], case["K"], case["F"]
    e = {"bf16": 2.0, "fp8": 1.0, "mxfp8": 1.0 + 1 / 32, "nvfp4": 0.5 + 1 / 16}[case["kind"]]
    if case["op"] == "gated":
        o = {"bf16": 2.0, "fp8": 1.0, "mxfp8": 1.0 + 1 / 32}[case["out"]]
        if case["keep"]:
            o += 4 + (2 if case["out"] != "bf16" else 0)
        return {"bytes": e * (T * K + 2 * F * K) + o * T * F, "flops": 4 * T * K * F}
    N = case["N"]
    b, f = e * (T * N + F * N) + 2 * T * 2 * F * 2, 2 * T * N * F
    if case["kind"] == "bf16":
        b, f = b + 2 * (2 * T * K + 2 * 2 * F * K), f + 2 * 4 * T * K * F
    return {"bytes": b, "flops": f}


# ---- inputs --------------------------------------------------------------------------------------

def _tiles(s, col_mult):
    """Scale bytes [R, C] -> the tensor-core layout: 128-row x 4-column tiles of 512 bytes."""
    R, C = s.shape
    rp, cp = -(-R // 128) * 128, -(-C // col_mult) * col_mult
    p = torch.zeros(rp, cp, dtype=torch.uint8, device=s.device)
    p[:R, :C] = s
    return p.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(t, R, C, col_mult):
    rp, cp = -(-R // 128) * 128, -(-C // col_mult) * col_mult
    return t.view(rp // 128, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp)[:R, :C]


def _quantized(t, kind, fmt="e4m3"):
    """The operand `t` (fp32) as the package's quantizers leave it."""
    if kind == "bf16":
        return dict(q=t.bfloat16())
    if kind == "fp8":
        s = FMAX[fmt] / t.abs().max()
        q = (t * s).clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)
        return dict(q=q, inv=(1.0 / s).reshape(1), fmt=fmt)
    R, C = t.shape
    if kind == "mxfp8":
        b = t.view(R, C // 32, 32)
        e = (torch.frexp(b.abs().amax(-1))[1] - 9).clamp(-127, 127)
        q = torch.ldexp(b, -e[..., None]).clamp(-448.0, 448.0).to(F8["e4m3"]).view(torch.uint8).view(R, C)
        return dict(q=q, s=_tiles((e + 127).to(torch.uint8), 4))
    b = t.view(R, C // 16, 16)
    enc = 2688.0 / t.abs().max()
    s = (b.abs().amax(-1) / 6.0 * enc).to(F8["e4m3"])
    v = b * torch.where(s.float() > 0, enc / s.float(), 0.0)[..., None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=t.device)
    c = (torch.bucketize(v.abs(), mids, out_int32=True).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)).view(R, C)
    return dict(q=c[:, 0::2] | (c[:, 1::2] << 4), s=_tiles(s.view(torch.uint8), 16), g=(1.0 / enc).reshape(1))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * std

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    u8, f32 = torch.uint8, torch.float32
    st = dict(case)
    if case["op"] in ("norm", "norm_bwd"):
        R, C, dt = case["rows"], case["cols"], DT[case["dtype"]]
        st["gamma"] = 1.0 + randn(C, std=0.1)
        hot = 1.0 + 20.0 * (torch.rand(C, generator=g, device=DEV) < 0.002)      # a few loud channels
        if case["op"] == "norm":
            st["x"] = randn(R, C).to(dt)
            st["res"] = (randn(R, C) * hot * 2.0).to(dt) if case["residual"] else None
            st["res_out"] = empty(R, C, dtype=dt) if case["residual"] else None
            st["y"], st["rsigma"] = (empty(R, C), empty(R, dtype=f32)) if case["keep"] else (None, None)
            st["q"] = empty(R, C, dtype=u8)
            if case["out"] == "fp8":
                st["scale"] = torch.full((1,), FMAX[case["fmt"]] / 6.5, device=DEV)   # an earlier step's amax
                st["amax"], st["inv"] = empty(1, dtype=f32), empty(1, dtype=f32)
            else:
                st["s"] = empty(-(-R // 128) * 128 * (-(-C // 128) * 4), dtype=u8)
            return st
        s = randn(R, C) * hot * 2.0
        st["s"] = s.to(dt)
        st["rsigma"] = torch.rsqrt(st["s"].float().square().mean(-1) + EPS)
        st["dy"] = randn(R, C, std=1e-3).bfloat16()
        st["dres"] = randn(R, C, std=1e-3).to(dt) if case["residual"] else None
        st["dx"], st["dgamma"] = empty(R, C, dtype=dt), empty(C, dtype=f32)
        st["ws"] = empty(512 * C, dtype=f32)      # at most 512 rows of partial column sums
        return st
    T, K, F, kind = case["T"], case["K"], case["F"], case["kind"]
    if case["op"] == "gated":
        st["x"] = _quantized(randn(T, K), kind)
        st["w"] = _quantized(randn(2 * F, K, std=1.28 / math.sqrt(K)), kind)
        out, keep = case["out"], case["keep"]
        st["gu"] = empty(T, 2 * F) if keep else None
        st["h"] = empty(T, F) if keep or out == "bf16" else None
        if out == "fp8":
            st["hq"], st["hscale"] = empty(T, F, dtype=u8), torch.full((1,), 448.0 / 12.0, device=DEV)
            st["amax"], st["inv"] = empty(1, dtype=f32), empty(1, dtype=f32)
        elif out == "mxfp8":
            st["hq"], st["hs"] = empty(T, F, dtype=u8), empty(-(-T // 128) * 128 * (F // 128 * 4), dtype=u8)
        return st
    N = case["N"]
    st["gu"] = randn(T, 2 * F, std=1.28).bfloat16()
    st["dy"] = _quantized(randn(T, N, std=1e-3), kind, "e5m2")
    w2 = randn(N, F, std=0.02)
    st["w2"] = _quantized(w2 if kind == "bf16" else w2.t().contiguous(), kind)   # 8- and 4-bit copies: [F, N]
    st["dgu"] = empty(T, 2 * F)
    if kind == "bf16":
        st["x"] = randn(T, K).bfloat16()
        st["w"] = randn(2 * F, K, std=1.28 / math.sqrt(K)).bfloat16()
        st["dx"], st["dw"] = empty(T, K), empty(2 * F, K)
    return st


# ---- the plain forms -------------------------------------------------------------------------------

def _values(o, kind, R, C):
    """fp32 values of a quantized operand [R, C] (per-tensor scales left out: one factor at the end)."""
    if kind == "bf16":
        return o["q"].float()
    if kind == "fp8":
        return o["q"].view(F8[o["fmt"]]).float()
    if kind == "mxfp8":
        s = torch.exp2(_untile(o["s"], R, C // 32, 4).float() - 127.0)
        return (o["q"].view(F8["e4m3"]).float().view(R, C // 32, 32) * s[..., None]).view(R, C)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=o["q"].device)
    q = torch.stack((o["q"] & 15, o["q"] >> 4), -1).view(R, C).int()
    s = _untile(o["s"], R, C // 16, 16).contiguous().view(F8["e4m3"]).float()
    return (lut[q].view(R, C // 16, 16) * s[..., None]).view(R, C)


def _alpha(a, b, kind):
    return a["inv"] * b["inv"] if kind == "fp8" else a["g"] * b["g"] if kind == "nvfp4" else 1.0


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _to_fp8(v, scale, fmt):
    return (v * scale).clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt])


def _to_mx(v):
    """Blocks of 32: E4M3 codes and the tiled power-of-two scales."""
    R, C = v.shape
    b = v.view(R, C // 32, 32)
    e = (torch.frexp(b.abs().amax(-1))[1] - 9).clamp(-127, 127)
    e = torch.where((b == 0).all(-1), -127, e)
    q = torch.ldexp(b, -e[..., None]).clamp(-448.0, 448.0).to(F8["e4m3"]).view(R, C)
    return q, _tiles((e + 127).to(torch.uint8), 4).view(torch.float8_e8m0fnu)


def _plain_norm(st):
    s = st["x"].float()
    if st["res"] is not None:
        s = s + st["res"].float()
    rs = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    y = s * rs * st["gamma"]
    out = {}
    if st["res"] is not None:
        out["res_out"] = s.to(st["x"].dtype)
    if st["keep"]:
        out.update(y=y.bfloat16(), rsigma=rs[:, 0])
    if st["out"] == "fp8":
        out.update(q=_to_fp8(y, st["scale"], st["fmt"]), amax=y.abs().max().reshape(1), inv=1.0 / st["scale"])
    else:
        out["q"], out["s"] = _to_mx(y)
    return out


def _plain_norm_bwd(st):
    rs = st["rsigma"][:, None]
    dy, xhat = st["dy"].float(), st["s"].float() * rs
    dg = dy * st["gamma"]
    dx = rs * (dg - xhat * (dg * xhat).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return dict(dx=dx.to(st["s"].dtype), dgamma=(dy * xhat).sum(0))


def _plain_gated(st):
    T, K, F, kind = st["T"], st["K"], st["F"], st["kind"]
    gu = _values(st["x"], kind, T, K) @ _values(st["w"], kind, 2 * F, K).t()
    gu = gu * _alpha(st["x"], st["w"], kind)
    h = _act(gu[:, :F], st["act"]) * gu[:, F:]
    out = {}
    if st["gu"] is not None:
        out["gu"] = gu.bfloat16()
    if st["h"] is not None:
        out["h"] = h.bfloat16()
    if st["out"] == "fp8":
        out.update(hq=_to_fp8(h, st["hscale"], "e4m3"), amax=h.abs().max().reshape(1), inv=1.0 / st["hscale"])
    elif st["out"] == "mxfp8":
        out["hq"], out["hs"] = _to_mx(h)
    return out


def _plain_gated_bwd(st):
    T, F, N, kind = st["T"], st["F"], st["N"], st["kind"]
    w2 = st["w2"]["q"].float() if kind == "bf16" else _values(st["w2"], kind, F, N).t()
    dh = _values(st["dy"], kind, T, N) @ w2 * _alpha(st["dy"], st["w2"], kind)
    g, u = st["gu"][:, :F].float(), st["gu"][:, F:].float()
    dgu = torch.cat((dh * u * _act_grad(g, st["act"]), dh * _act(g, st["act"])), 1)
    out = dict(dgu=dgu.bfloat16())
    if kind == "bf16":
        out.update(dx=(dgu @ st["w"].float()).bfloat16(), dw=(dgu.t() @ st["x"].float()).bfloat16())
    return out


# ---- the package's calls ---------------------------------------------------------------------------

def _own(st):
    import nvfp4_precision_transformer_gb300 as te
    op, out = st["op"], {}
    if op == "norm":
        fmt = te.E4M3 if st["fmt"] == "e4m3" else te.E5M2
        if st["out"] == "fp8":
            te.te_rmsnorm_fp8(st["x"], st["gamma"], EPS, fmt, st["scale"], st["q"], residual=st["res"],
                              res_out=st["res_out"], y=st["y"], rsigma=st["rsigma"], amax_out=st["amax"],
                              scale_inv_out=st["inv"])
            out.update(q=st["q"].view(F8[st["fmt"]]), amax=st["amax"], inv=st["inv"])
        else:
            te.te_rmsnorm_mxfp8(st["x"], st["gamma"], EPS, st["q"], st["s"], residual=st["res"], res_out=st["res_out"],
                                y=st["y"], rsigma=st["rsigma"])
            out.update(q=st["q"].view(F8["e4m3"]), s=st["s"].view(torch.float8_e8m0fnu))
        if st["res"] is not None:
            out["res_out"] = st["res_out"]
        if st["keep"]:
            out.update(y=st["y"], rsigma=st["rsigma"])
        return out
    if op == "norm_bwd":
        te.te_rmsnorm_bwd(st["dy"], st["s"], st["gamma"], st["rsigma"], st["dx"], st["dgamma"], st["ws"],
                          dres=st["dres"])
        return dict(dx=st["dx"], dgamma=st["dgamma"])
    kind, act = st["kind"], te.ACT_SILU if st["act"] == "silu" else te.ACT_GELU
    if op == "gated":
        x, w, h, gu = st["x"], st["w"], st["h"], st["gu"]
        if kind == "bf16":
            te.te_gated_gemm_bf16(x["q"], w["q"], act, h=h, gu=gu)
        elif kind == "fp8":
            more = dict(q_h=st["hq"], h_fmt=te.E4M3, h_scale=st["hscale"], h_amax=st["amax"],
                        h_scale_inv=st["inv"]) if st["out"] == "fp8" else {}
            te.te_gated_gemm_fp8(x["q"], te.E4M3, w["q"], te.E4M3, x["inv"], w["inv"], act, h=h, gu=gu, **more)
        elif kind == "mxfp8":
            more = dict(q_h=st["hq"], s_h=st["hs"]) if st["out"] == "mxfp8" else {}
            te.te_gated_gemm_mxfp8(x["q"], x["s"], w["q"], w["s"], act, h=h, gu=gu, **more)
        else:
            te.te_gated_gemm_nvfp4(x["q"], x["s"], x["g"], w["q"], w["s"], w["g"], act, h=h, gu=gu)
        if gu is not None:
            out["gu"] = gu
        if h is not None:
            out["h"] = h
        if st["out"] == "fp8":
            out.update(hq=st["hq"].view(F8["e4m3"]), amax=st["amax"], inv=st["inv"])
        elif st["out"] == "mxfp8":
            out.update(hq=st["hq"].view(F8["e4m3"]), hs=st["hs"].view(torch.float8_e8m0fnu))
        return out
    dy, w2 = st["dy"], st["w2"]
    if kind == "bf16":
        te.te_gated_bwd_bf16(st["x"], st["w"], w2["q"], dy["q"], st["gu"], act, st["dgu"], st["dx"], st["dw"])
        return dict(dgu=st["dgu"], dx=st["dx"], dw=st["dw"])
    if kind == "fp8":
        te.te_gated_dgrad_fp8(dy["q"], te.E5M2, w2["q"], te.E4M3, dy["inv"], w2["inv"], st["gu"], act, st["dgu"])
    elif kind == "mxfp8":
        te.te_gated_dgrad_mxfp8(dy["q"], dy["s"], w2["q"], w2["s"], st["gu"], act, st["dgu"])
    else:
        te.te_gated_dgrad_nvfp4(dy["q"], dy["s"], dy["g"], w2["q"], w2["s"], w2["g"], st["gu"], act, st["dgu"])
    return dict(dgu=st["dgu"])


def run(st):
    if own:
        return _own(st)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gated": _plain_gated,
            "gated_bwd": _plain_gated_bwd}[st["op"]](st)


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _f64(o, kind, R, C):
    """The operand's values in 64 bits, its per-tensor scale included."""
    q = o["q"]
    if kind == "bf16":
        return q.double()
    if kind == "fp8":
        return q.view(F8[o["fmt"]]).double() * o["inv"].double()
    block, mult = (32, 4) if kind == "mxfp8" else (16, 16)
    n = C // block
    r = torch.arange(R, device=q.device)[:, None]
    j = torch.arange(n, device=q.device)[None, :]
    at = ((r // 128) * (-(-n // mult) * mult // 4) + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    b = o["s"][at]
    if kind == "mxfp8":
        v, s = q.view(F8["e4m3"]).double(), torch.pow(2.0, b.double() - 127.0)
    else:
        s = b.view(F8["e4m3"]).double() * o["g"].double()
        n4 = torch.empty(R, C, dtype=torch.uint8, device=q.device)
        n4[:, 0::2], n4[:, 1::2] = q & 15, q >> 4
        m = (n4 & 7).double()                                            # E2M1: 0 .5 1 1.5 2 3 4 6
        v = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8)) * torch.where(n4 > 7, -1.0, 1.0).double()
    return v * s.repeat_interleave(block, 1)


def _mx64(v):
    R, C = v.shape
    b = v.reshape(R, C // 32, 32)
    top = b.abs().max(-1).values
    e = torch.where(top > 0, torch.floor(torch.log2(top)) - 8, -127.0).clamp(-127, 127)
    q = (b / torch.pow(2.0, e)[..., None]).clamp(-448, 448).reshape(R, C)
    return q, torch.pow(2.0, _tiles((e + 127).to(torch.uint8), 4).double() - 127.0)


def _gates64(g, act):
    """(act(g), act'(g)) in 64 bits."""
    if act == "silu":
        z = torch.exp(-g)
        return g / (1 + z), (1 + z + g * z) / (1 + z) ** 2
    c, d = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * g * (1 + d * g ** 2))
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * c * (1 + 3 * d * g ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    out = {}
    if case["op"] == "norm":
        s = st["x"].double() + (st["res"].double() if st["res"] is not None else 0.0)
        inv = 1.0 / torch.sqrt((s ** 2).sum(1) / case["cols"] + EPS)
        y = s * inv[:, None] * st["gamma"].double()
        if st["res"] is not None:
            out["res_out"] = s
        if case["keep"]:
            out.update(y=y, rsigma=inv)
        if case["out"] == "fp8":
            top = FMAX[case["fmt"]]
            out.update(q=(y * st["scale"].double()).clamp(-top, top), amax=y.abs().max().reshape(1),
                       inv=1.0 / st["scale"].double())
        else:
            out["q"], out["s"] = _mx64(y)
        return out
    if case["op"] == "norm_bwd":
        r, dy, s = st["rsigma"].double()[:, None], st["dy"].double(), st["s"].double()
        p = dy * st["gamma"].double()
        dx = r * p - s * r ** 3 * ((p * s).sum(1, keepdim=True) / case["cols"])
        if st["dres"] is not None:
            dx = dx + st["dres"].double()
        return dict(dx=dx, dgamma=(dy * s * r).sum(0))
    T, K, F, kind = case["T"], case["K"], case["F"], case["kind"]
    if case["op"] == "gated":
        x, w = _f64(st["x"], kind, T, K), _f64(st["w"], kind, 2 * F, K)
        g, u = x @ w[:F].t(), x @ w[F:].t()
        h = _gates64(g, case["act"])[0] * u
        if st["gu"] is not None:
            out["gu"] = torch.cat((g, u), 1)
        if st["h"] is not None:
            out["h"] = h
        if case["out"] == "fp8":
            out.update(hq=(h * st["hscale"].double()).clamp(-448, 448), amax=h.abs().max().reshape(1),
                       inv=1.0 / st["hscale"].double())
        elif case["out"] == "mxfp8":
            out["hq"], out["hs"] = _mx64(h)
        return out
    N = case["N"]
    dy = _f64(st["dy"], kind, T, N)
    dh = dy @ (st["w2"]["q"].double() if kind == "bf16" else _f64(st["w2"], kind, F, N).t())
    a, da = _gates64(st["gu"][:, :F].double(), case["act"])
    dg, du = dh * st["gu"][:, F:].double() * da, dh * a
    out["dgu"] = torch.cat((dg, du), 1)
    if kind == "bf16":
        w, x = st["w"].double(), st["x"].double()
        out.update(dx=dg @ w[:F] + du @ w[F:], dw=torch.cat((dg.t() @ x, du.t() @ x), 0))
    return out
