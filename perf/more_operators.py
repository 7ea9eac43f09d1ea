"""LayerNorm and the linear with bias, activation and residual: measured cases and their plain forms.

Four passes of the pre-norm feed-forward half of a layer (norm, up projection with bias and activation, down
projection with bias and residual), each in the formats of this package (FP8 with one scale a tensor, MXFP8,
NVFP4) or in BF16:

  ln       s = x + residual;  y = (s - mu) * rsigma * gamma + beta, and y in 8 bits with scales
  ln_bwd   the gradients of x (and of the residual, the same tensor), of gamma and of beta
  act      z = x w^T + bias;  y = act(z) + residual, or act(z) in 8 bits; z where the backward pass keeps it
  act_bwd  from the gradient dy of act(z) w2^T: the gradients of z and of the bias, and (BF16) of x and w

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
        # decoding one token with the FP8 recipe: the norm before the feed-forward half
        dict(name="ln_fp8_token", op="ln", rows=1, cols=4096, dtype="bf16", residual=True, out="fp8", fmt="e4m3",
             keep=False),
        # the norm of a training layer under MXFP8: everything that its backward pass needs is kept
        dict(name="ln_mxfp8_layer", op="ln", rows=15872, cols=4096, dtype="bf16", residual=True, out="mxfp8",
             fmt="e4m3", keep=True),
        # a tutorial-sized model in training with an odd number of rows and an fp32 residual stream
        dict(name="ln_bwd_fp32_odd", op="ln_bwd", rows=1023, cols=768, dtype="fp32", residual=True),
        # the training layer's norm, with the gradient that comes down the residual stream
        dict(name="ln_bwd_layer", op="ln_bwd", rows=15872, cols=4096, dtype="bf16", residual=True),
        # decoding one token: the down projection, whose result goes onto the residual stream
        dict(name="act_bf16_token", op="act", kind="bf16", T=1, K=16384, N=4096, act="none", bias=True, residual=True,
             out="bf16", keep=False),
        # a batch of requests that decode together, FP8 weights: the up projection
        dict(name="act_fp8_batch", op="act", kind="fp8", T=24, K=4096, N=16384, act="gelu", bias=True, residual=False,
             out="fp8", keep=False),
        # one sequence of training or prefill under MXFP8, a ragged token count, pre-activations kept
        dict(name="act_mxfp8_sequence", op="act", kind="mxfp8", T=509, K=4096, N=16384, act="gelu", bias=True,
             residual=False, out="mxfp8", keep=True),
        # the training layer under FP8: act(z) leaves in FP8 for the down projection, z is kept
        dict(name="act_fp8_layer", op="act", kind="fp8", T=15872, K=4096, N=16384, act="gelu", bias=True,
             residual=False, out="fp8", keep=True),
        # the training layer's down projection under NVFP4, onto the residual stream
        dict(name="act_nvfp4_down", op="act", kind="nvfp4", T=15872, K=16384, N=4096, act="none", bias=True,
             residual=True, out="bf16", keep=False),
        # a tutorial-sized backward pass with a ragged token count
        dict(name="act_bwd_bf16_odd", op="act_bwd", kind="bf16", T=1001, K=768, F=2048, N=768, act="relu"),
        # eight sequences under MXFP8: the up projection's pre-activations and bias
        dict(name="act_bwd_mxfp8", op="act_bwd", kind="mxfp8", T=4096, K=4096, F=16384, N=4096, act="gelu"),
        # the training layer's backward pass: the largest case
        dict(name="act_bwd_bf16_layer", op="act_bwd", kind="bf16", T=15872, K=4096, F=16384, N=4096, act="gelu"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _mult(rng, lo, hi, m):
    return max(1, round(_log(rng, lo, hi) / m)) * m


def draw(rng):
    op = rng.choice(("ln", "ln", "ln_bwd", "act", "act", "act", "act", "act_bwd", "act_bwd"))
    if op in ("ln", "ln_bwd"):
        out = rng.choice(("fp8", "mxfp8"))
        cols = _mult(rng, 64, 16384, 32 if out == "mxfp8" and op == "ln" else 16)
        rows = min(int(_log(rng, 1, 16384)), 15872 * 4096 // cols)
        case = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(("bf16", "fp32")), residual=rng.random() < 0.75)
        if op == "ln":
            case.update(out=out, fmt=rng.choice(("e4m3", "e5m2")) if out == "fp8" else "e4m3", keep=rng.random() < 0.5)
        return case
    kind = rng.choice(("bf16", "fp8", "mxfp8", "nvfp4"))
    block = 32 if kind in ("mxfp8", "nvfp4") else 16
    T = int(_log(rng, 1, 15872))
    K = _mult(rng, 64, 16384, block)
    N = _mult(rng, 64, 16384, 32 if kind == "mxfp8" else 16)
    while T * K * N > 15872 * 4096 * 16384:
        T //= 2
    case = dict(op=op, kind=kind, T=T, act=rng.choice(("none", "relu", "silu", "gelu")))
    if op == "act":
        out = rng.choice(("bf16", "fp32", kind)) if kind in ("fp8", "mxfp8") else rng.choice(("bf16", "bf16", "fp32"))
        case.update(K=K, N=N, out=out, bias=rng.random() < 0.75,
                    residual=out in ("bf16", "fp32") and rng.random() < 0.5, keep=rng.random() < 0.5)
    else:
        case.update(K=K, F=N, N=K)
    return case


def work(case):
    if case["op"] in ("ln", "ln_bwd"):
        n, e = case["rows"] * case["cols"], 4 if case["dtype"] == "fp32" else 2
        r = 1 if case["residual"] else 0
        if case["op"] == "ln":
            b = n * (e + 2 * e * r + 1 + (2 if case["keep"] else 0)) + (n // 32 if case["out"] == "mxfp8" else 0)
            return {"bytes": b + 8 * case["cols"] + (8 * case["rows"] if case["keep"] else 0), "flops": 8 * n}
        return {"bytes": n * (2 + 2 * e + e * r) + 12 * case["cols"] + 8 * case["rows"], "flops": 15 * n}
    T, K = case["T"], case["K"]
    e = {"bf16": 2.0, "fp8": 1.0, "mxfp8": 1.0 + 1 / 32, "nvfp4": 0.5 + 1 / 16}[case["kind"]]
    if case["op"] == "act":
        N, out = case["N"], case["out"]
        o = {"bf16": 2.0, "fp32": 4.0, "fp8": 1.0, "mxfp8": 1.0 + 1 / 32}[out] * (2 if case["residual"] else 1)
        if case["keep"]:
            o += 2 + (2 if out in ("fp8", "mxfp8") else 0)
        return {"bytes": e * (T * K + N * K) + o * T * N + (4 * N if case["bias"] else 0), "flops": 2 * T * K * N}
    F, N = case["F"], case["N"]
    b, f = e * (T * N + F * N) + 2 * T * F * (1 if case["act"] == "none" else 2) + 4 * F, 2 * T * N * F
    if case["kind"] == "bf16":
        b, f = b + 2 * (2 * T * K + 2 * F * K), f + 4 * T * K * F
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
    if case["op"] in ("ln", "ln_bwd"):
        R, C, dt = case["rows"], case["cols"], DT[case["dtype"]]
        st["gamma"], st["beta"] = 1.0 + randn(C, std=0.1), randn(C, std=0.1)
        hot = 1.0 + 20.0 * (torch.rand(C, generator=g, device=DEV) < 0.002)      # a few loud channels
        shift = randn(C, std=0.5)                                                # channels with a mean of their own
        if case["op"] == "ln":
            st["x"] = randn(R, C).to(dt)
            st["res"] = (randn(R, C) * hot * 2.0 + shift).to(dt) if case["residual"] else None
            st["res_out"] = empty(R, C, dtype=dt) if case["residual"] else None
            st["y"], st["mu"], st["rsigma"] = ((empty(R, C), empty(R, dtype=f32), empty(R, dtype=f32)) if case["keep"]
                                               else (None, None, None))
            st["q"] = empty(R, C, dtype=u8)
            if case["out"] == "fp8":
                st["scale"] = torch.full((1,), FMAX[case["fmt"]] / 6.5, device=DEV)   # an earlier step's amax
                st["amax"], st["inv"] = empty(1, dtype=f32), empty(1, dtype=f32)
            else:
                st["s"] = empty(-(-R // 128) * 128 * (-(-C // 128) * 4), dtype=u8)
            return st
        st["s"] = (randn(R, C) * hot * 2.0 + shift).to(dt)
        st["mu"] = st["s"].float().mean(-1)
        st["rsigma"] = torch.rsqrt((st["s"].float() - st["mu"][:, None]).square().mean(-1) + EPS)
        st["dy"] = randn(R, C, std=1e-3).bfloat16()
        st["dres"] = randn(R, C, std=1e-3).to(dt) if case["residual"] else None
        st["dx"], st["dgamma"], st["dbeta"] = empty(R, C, dtype=dt), empty(C, dtype=f32), empty(C, dtype=f32)
        st["ws"] = empty(2 * min(R, 512) * C, dtype=f32)      # at most 512 rows of two partial column sums
        return st
    T, K, kind = case["T"], case["K"], case["kind"]
    if case["op"] == "act":
        N, out, keep = case["N"], case["out"], case["keep"]
        st["x"] = _quantized(randn(T, K), kind)
        st["w"] = _quantized(randn(N, K, std=1.28 / math.sqrt(K)), kind)
        st["b"] = randn(N, std=0.1) if case["bias"] else None
        ydt = f32 if out == "fp32" else torch.bfloat16
        st["res"] = randn(T, N, std=2.0).to(ydt) if case["residual"] else None
        st["z"] = empty(T, N) if keep else None
        st["y"] = empty(T, N, dtype=ydt) if keep or out in ("bf16", "fp32") else None
        if out == "fp8":
            st["yq"], st["yscale"] = empty(T, N, dtype=u8), torch.full((1,), 448.0 / 7.0, device=DEV)
            st["amax"], st["inv"] = empty(1, dtype=f32), empty(1, dtype=f32)
        elif out == "mxfp8":
            st["yq"], st["ys"] = empty(T, N, dtype=u8), empty(-(-T // 128) * 128 * (-(-N // 128) * 4), dtype=u8)
        return st
    F, N = case["F"], case["N"]
    st["z"] = randn(T, F, std=1.28).bfloat16() if case["act"] != "none" else None
    st["dy"] = _quantized(randn(T, N, std=1e-3), kind, "e5m2")
    w2 = randn(N, F, std=0.02)
    st["w2"] = _quantized(w2 if kind == "bf16" else w2.t().contiguous(), kind)   # 8- and 4-bit copies: [F, N]
    st["dz"], st["dbias"] = empty(T, F), empty(F, dtype=f32)
    st["ws"] = empty(-(-T // 32) * F, dtype=f32)      # a row of partial sums for each 32 tokens
    if kind == "bf16":
        st["x"] = randn(T, K).bfloat16()
        st["w"] = randn(F, K, std=1.28 / math.sqrt(K)).bfloat16()
        st["dx"], st["dw"] = empty(T, K), empty(F, K)
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


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


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


def _plain_ln(st):
    s = st["x"].float()
    if st["res"] is not None:
        s = s + st["res"].float()
    mu = s.mean(-1, keepdim=True)
    d = s - mu
    rs = torch.rsqrt(d.square().mean(-1, keepdim=True) + EPS)
    y = d * rs * st["gamma"] + st["beta"]
    out = {}
    if st["res"] is not None:
        out["res_out"] = s.to(st["x"].dtype)
    if st["keep"]:
        out.update(y=y.bfloat16(), mu=mu[:, 0], rsigma=rs[:, 0])
    if st["out"] == "fp8":
        out.update(q=_to_fp8(y, st["scale"], st["fmt"]), amax=y.abs().max().reshape(1), inv=1.0 / st["scale"])
    else:
        out["q"], out["s"] = _to_mx(y)
    return out


def _plain_ln_bwd(st):
    rs = st["rsigma"][:, None]
    dy, xhat = st["dy"].float(), (st["s"].float() - st["mu"][:, None]) * rs
    p = dy * st["gamma"]
    dx = rs * (p - p.mean(-1, keepdim=True) - xhat * (p * xhat).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return dict(dx=dx.to(st["s"].dtype), dgamma=(dy * xhat).sum(0), dbeta=dy.sum(0))


def _plain_act(st):
    T, K, N, kind = st["T"], st["K"], st["N"], st["kind"]
    z = _values(st["x"], kind, T, K) @ _values(st["w"], kind, N, K).t()
    z = z * _alpha(st["x"], st["w"], kind)
    if st["b"] is not None:
        z = z + st["b"]
    a = _act(z, st["act"])
    out = {}
    if st["z"] is not None:
        out["z"] = z.bfloat16()
    if st["y"] is not None:
        out["y"] = (a if st["res"] is None else a + st["res"].float()).to(st["y"].dtype)
    if st["out"] == "fp8":
        out.update(yq=_to_fp8(a, st["yscale"], "e4m3"), amax=a.abs().max().reshape(1), inv=1.0 / st["yscale"])
    elif st["out"] == "mxfp8":
        out["yq"], out["ys"] = _to_mx(a)
    return out


def _plain_act_bwd(st):
    T, F, N, kind = st["T"], st["F"], st["N"], st["kind"]
    w2 = st["w2"]["q"].float() if kind == "bf16" else _values(st["w2"], kind, F, N).t()
    dz = _values(st["dy"], kind, T, N) @ w2 * _alpha(st["dy"], st["w2"], kind)
    if st["z"] is not None:
        dz = dz * _act_grad(st["z"].float(), st["act"])
    out = dict(dz=dz.bfloat16(), dbias=dz.sum(0))
    if kind == "bf16":
        out.update(dx=(dz @ st["w"].float()).bfloat16(), dw=(dz.t() @ st["x"].float()).bfloat16())
    return out


# ---- the package's calls ---------------------------------------------------------------------------

def _own(st):
    import nvfp4_precision_transformer_gb300 as te
    op, out = st["op"], {}
    if op == "ln":
        common = dict(residual=st["res"], res_out=st["res_out"], y=st["y"], mu=st["mu"], rsigma=st["rsigma"])
        if st["out"] == "fp8":
            fmt = te.E4M3 if st["fmt"] == "e4m3" else te.E5M2
            te.te_add_layernorm_fp8(st["x"], st["gamma"], st["beta"], EPS, fmt, st["scale"], st["q"],
                                    amax_out=st["amax"], scale_inv_out=st["inv"], **common)
            out.update(q=st["q"].view(F8[st["fmt"]]), amax=st["amax"], inv=st["inv"])
        else:
            te.te_add_layernorm_mxfp8(st["x"], st["gamma"], st["beta"], EPS, st["q"], st["s"], **common)
            out.update(q=st["q"].view(F8["e4m3"]), s=st["s"].view(torch.float8_e8m0fnu))
        if st["res"] is not None:
            out["res_out"] = st["res_out"]
        if st["keep"]:
            out.update(y=st["y"], mu=st["mu"], rsigma=st["rsigma"])
        return out
    if op == "ln_bwd":
        te.te_layernorm_bwd(st["dy"], st["s"], st["gamma"], st["mu"], st["rsigma"], st["dx"], st["dgamma"], st["dbeta"],
                            st["ws"], dres=st["dres"])
        return dict(dx=st["dx"], dgamma=st["dgamma"], dbeta=st["dbeta"])
    kind = st["kind"]
    act = {"none": te.ACT_NONE, "relu": te.ACT_RELU, "silu": te.ACT_SILU, "gelu": te.ACT_GELU}[st["act"]]
    if op == "act":
        x, w, more = st["x"], st["w"], dict(y=st["y"], z=st["z"], bias=st["b"], residual=st["res"])
        if kind == "bf16":
            te.te_act_gemm_bf16(x["q"], w["q"], act, **more)
        elif kind == "fp8":
            if st["out"] == "fp8":
                more.update(q=st["yq"], q_fmt=te.E4M3, q_scale=st["yscale"], q_amax=st["amax"], q_scale_inv=st["inv"])
            te.te_act_gemm_fp8(x["q"], te.E4M3, w["q"], te.E4M3, x["inv"], w["inv"], act, **more)
        elif kind == "mxfp8":
            if st["out"] == "mxfp8":
                more.update(q=st["yq"], s_q=st["ys"])
            te.te_act_gemm_mxfp8(x["q"], x["s"], w["q"], w["s"], act, **more)
        else:
            te.te_act_gemm_nvfp4(x["q"], x["s"], x["g"], w["q"], w["s"], w["g"], act, **more)
        if st["z"] is not None:
            out["z"] = st["z"]
        if st["y"] is not None:
            out["y"] = st["y"]
        if st["out"] == "fp8":
            out.update(yq=st["yq"].view(F8["e4m3"]), amax=st["amax"], inv=st["inv"])
        elif st["out"] == "mxfp8":
            out.update(yq=st["yq"].view(F8["e4m3"]), ys=st["ys"].view(torch.float8_e8m0fnu))
        return out
    dy, w2, more = st["dy"], st["w2"], dict(dbias=st["dbias"], workspace=st["ws"])
    if kind == "bf16":
        te.te_act_bwd_bf16(st["x"], st["w"], w2["q"], dy["q"], st["z"], act, st["dz"], dx=st["dx"], dw=st["dw"], **more)
        return dict(dz=st["dz"], dbias=st["dbias"], dx=st["dx"], dw=st["dw"])
    if kind == "fp8":
        te.te_act_dgrad_fp8(dy["q"], te.E5M2, w2["q"], te.E4M3, dy["inv"], w2["inv"], st["z"], act, st["dz"], **more)
    elif kind == "mxfp8":
        te.te_act_dgrad_mxfp8(dy["q"], dy["s"], w2["q"], w2["s"], st["z"], act, st["dz"], **more)
    else:
        te.te_act_dgrad_nvfp4(dy["q"], dy["s"], dy["g"], w2["q"], w2["s"], w2["g"], st["z"], act, st["dz"], **more)
    return dict(dz=st["dz"], dbias=st["dbias"])


def run(st):
    if own:
        return _own(st)
    return {"ln": _plain_ln, "ln_bwd": _plain_ln_bwd, "act": _plain_act, "act_bwd": _plain_act_bwd}[st["op"]](st)


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


def _act64(z, act):
    """(act(z), act'(z)) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).double()
    if act == "silu":
        t = torch.exp(-z)
        return z / (1 + t), (1 + t + z * t) / (1 + t) ** 2
    c, d = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * z * (1 + d * z ** 2))
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t ** 2) * c * (1 + 3 * d * z ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    out = {}
    if case["op"] == "ln":
        s = st["x"].double() + (st["res"].double() if st["res"] is not None else 0.0)
        n = case["cols"]
        mu = s.sum(1) / n
        c = s - mu[:, None]
        inv = 1.0 / torch.sqrt((c ** 2).sum(1) / n + EPS)
        y = c * inv[:, None] * st["gamma"].double() + st["beta"].double()
        if st["res"] is not None:
            out["res_out"] = s
        if case["keep"]:
            out.update(y=y, mu=mu, rsigma=inv)
        if case["out"] == "fp8":
            top = FMAX[case["fmt"]]
            out.update(q=(y * st["scale"].double()).clamp(-top, top), amax=y.abs().max().reshape(1),
                       inv=1.0 / st["scale"].double())
        else:
            out["q"], out["s"] = _mx64(y)
        return out
    if case["op"] == "ln_bwd":
        n, r, dy = case["cols"], st["rsigma"].double()[:, None], st["dy"].double()
        c = st["s"].double() - st["mu"].double()[:, None]
        p = dy * st["gamma"].double()
        dx = r * (p - p.sum(1, keepdim=True) / n) - c * r ** 3 * ((p * c).sum(1, keepdim=True) / n)
        if st["dres"] is not None:
            dx = dx + st["dres"].double()
        return dict(dx=dx, dgamma=(dy * c * r).sum(0), dbeta=dy.sum(0))
    T, K, kind = case["T"], case["K"], case["kind"]
    if case["op"] == "act":
        N = case["N"]
        z = _f64(st["x"], kind, T, K) @ _f64(st["w"], kind, N, K).t()
        if st["b"] is not None:
            z = z + st["b"].double()
        a = _act64(z, case["act"])[0]
        if st["z"] is not None:
            out["z"] = z
        if st["y"] is not None:
            out["y"] = a if st["res"] is None else a + st["res"].double()
        if case["out"] == "fp8":
            out.update(yq=(a * st["yscale"].double()).clamp(-448, 448), amax=a.abs().max().reshape(1),
                       inv=1.0 / st["yscale"].double())
        elif case["out"] == "mxfp8":
            out["yq"], out["ys"] = _mx64(a)
        return out
    F, N = case["F"], case["N"]
    dz = _f64(st["dy"], kind, T, N) @ (st["w2"]["q"].double() if kind == "bf16" else _f64(st["w2"], kind, F, N).t())
    if st["z"] is not None:
        dz = dz * _act64(st["z"].double(), case["act"])[1]
    out = dict(dz=dz, dbias=dz.sum(0))
    if kind == "bf16":
        out.update(dx=dz @ st["w"].double(), dw=dz.t() @ st["x"].double())
    return out
