"""The feed-forward half of a pre-norm transformer layer with one activation (te.LayerNormMLP's place), as sequences
of C-ABI calls.

    s = x + residual
    n = LayerNorm(s) * gamma + beta
    h = act(n W1^T + b1)                    w1 [F, K]
    y = s + h W2^T + b2                     w2 [K, F]

and its backward pass.  The recipes are those of ``gated``: bf16, fp8_delayed (HYBRID) and mxfp8; the norm writes n
and the up projection writes h in 8 bits for the GEMM after it.

Everything here is marshalling: device buffers (torch allocations) and the order of launches; all arithmetic runs in
libte_gb300.so.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .gated import RECIPES, _Block, _need16

FWD_SLOTS = ("n", "w1", "h", "w2")
BWD_SLOTS = ("dy", "dz")
CAST_ELEMENTS = 1 << 34     # a quantizer takes fewer


class MLP(_Block):
    """Device buffers of one feed-forward block for ``tokens`` tokens, its forward and backward pass.

    ``forward(x, residual)`` returns y, the stream that the next block reads; ``residual`` may be None (x is the stream).
    ``backward(dy)`` takes its gradient and leaves ``dx`` (the gradient of x and of residual alike), ``dgamma``,
    ``dbeta``, ``dw1``, ``db1``, ``dw2`` and ``db2``.

    x, residual and dy are contiguous bf16 [tokens, K], tokens, K and F multiples of 16 (32 in MXFP8), K at most 16384; w1
    and w2 bf16, or fp32 where the recipe quantizes them; gamma, beta, b1, b2 fp32; all on 16-byte boundaries.  Anything
    else is refused before the first launch.
    Where residual is None, x itself is what the backward pass reads as s: it has to keep its values until then."""

    def __init__(self, gamma: torch.Tensor, beta: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor,
                 b2: torch.Tensor, tokens: int, recipe: str = "bf16", act: int = L.ACT_GELU, eps: float = 1e-5,
                 history_len: int = 16):
        if recipe not in RECIPES:
            raise ValueError(f"recipe {recipe!r} is none of {RECIPES}")
        if w1.dim() != 2 or w2.shape != (w1.shape[1], w1.shape[0]):
            raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} are not [F, K] and [K, F]")
        F, K = w1.shape
        step = 32 if recipe == "mxfp8" else 16
        if tokens <= 0 or tokens % step or K % step or F % step:
            raise ValueError(f"{tokens} tokens, K {K} and F {F} are not multiples of {step}")
        self._check_norm(K, eps)
        # (dy, and under the other recipes h and dz, go through the quantizers)
        if tokens * (K if recipe == "bf16" else max(K, F)) >= CAST_ELEMENTS:
            raise ValueError(f"{tokens} tokens of K {K} and F {F} are more than a quantizer takes, {CAST_ELEMENTS - 1} elements")
        if act not in (L.ACT_NONE, L.ACT_RELU, L.ACT_SILU, L.ACT_GELU):
            raise ValueError(f"act {act} is no activation")
        self.gamma, self.beta, self.w1, self.b1, self.w2, self.b2 = gamma, beta, w1, b1, w2, b2
        self.T, self.K, self.F, self.recipe, self.act, self.eps = tokens, K, F, recipe, act, eps
        self._check_weights("MLP", L._device())
        dev, T = w1.device, tokens
        bf, f32 = (dict(dtype=t, device=dev) for t in (torch.bfloat16, torch.float32))
        self._s, self.n, self.h, self.z = (torch.empty(T, c, **bf) for c in (K, K, F, F))
        self.y, self.dn, self.dx, self.dz = (torch.empty(T, c, **bf) for c in (K, K, K, F))
        self.dw1, self.dw2 = torch.empty(F, K, **bf), torch.empty(K, F, **bf)
        self.mu, self.rsigma = torch.empty(T, **f32), torch.empty(T, **f32)
        self.dgamma, self.dbeta, self.db1, self.db2 = (torch.empty(c, **f32) for c in (K, K, F, K))
        self.one = torch.ones(1, **f32)
        # one workspace: its users run one after the other
        self.workspace = torch.empty(max(L.te_layernorm_bwd_workspace_bytes(T, K), L.te_act_dbias_workspace_bytes(T, F),
                                         L.te_dbias_workspace_bytes(T, K)) // 4, **f32)
        self._allocate({"n": (T, K), "w1": (F, K), "h": (T, F), "w2": (K, F), "dy": (T, K), "dz": (T, F)},
                       FWD_SLOTS, BWD_SLOTS, history_len, dev)
        self.s = None

    def _check_weights(self, fn: str, dev: int) -> None:
        """Before the first launch of a pass, whose calls take addresses and sizes as they are."""
        weight = torch.bfloat16 if self.recipe == "bf16" else (torch.bfloat16, torch.float32)
        for name, dtype, shape in (("gamma", torch.float32, (self.K,)), ("beta", torch.float32, (self.K,)),
                                   ("w1", weight, (self.F, self.K)), ("b1", torch.float32, (self.F,)),
                                   ("w2", weight, (self.K, self.F)), ("b2", torch.float32, (self.K,))):
            _need16(fn, dev, name, getattr(self, name), dtype, shape)

    # ---- passes ----------------------------------------------------------------------------------
    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        E4, shape = L.E4M3, (self.T, self.K)
        fn, dev = "MLP.forward", L._device()
        self._check_weights(fn, dev)
        _need16(fn, dev, "x", x, torch.bfloat16, shape)
        _need16(fn, dev, "residual", residual, torch.bfloat16, shape, True)
        self.s = x if residual is None else self._s
        norm = dict(residual=residual, res_out=None if residual is None else self.s, y=self.n, mu=self.mu, rsigma=self.rsigma)
        up, down = dict(y=self.h, z=self.z, bias=self.b1), dict(y=self.y, bias=self.b2, residual=self.s)
        if self.recipe == "bf16":
            L.te_add_layernorm_fp8(x, self.gamma, self.beta, self.eps, E4, **norm)
            L.te_act_gemm_bf16(self.n, self.w1, self.act, **up)
            L.te_act_gemm_bf16(self.h, self.w2, L.ACT_NONE, **down)
            return self.y
        self._quantize("w1", self.w1, E4)
        self._quantize("w2", self.w2, E4)
        row = self.row
        if self.recipe == "mxfp8":
            srow = self.srow
            L.te_add_layernorm_mxfp8(x, self.gamma, self.beta, self.eps, row["n"], srow["n"], **norm)
            L.te_act_gemm_mxfp8(row["n"], srow["n"], row["w1"], srow["w1"], self.act, q=row["h"], s_q=srow["h"], **up)
            L.te_act_gemm_mxfp8(row["h"], srow["h"], row["w2"], srow["w2"], L.ACT_NONE, **down)
        else:
            s = self.slots
            L.te_add_layernorm_fp8(x, self.gamma, self.beta, self.eps, E4, s["n"][0], row["n"], amax_out=s["n"][2], **norm)
            L.te_act_gemm_fp8(row["n"], E4, row["w1"], E4, s["n"][1], s["w1"][1], self.act, q=row["h"], q_fmt=E4,
                              q_scale=s["h"][0], q_amax=s["h"][2], **up)
            L.te_act_gemm_fp8(row["h"], E4, row["w2"], E4, s["h"][1], s["w2"][1], L.ACT_NONE, **down)
        return self.y

    def backward(self, dy: torch.Tensor) -> None:
        E4, E5, MN = L.E4M3, L.E5M2, L.MN_MAJOR
        fn, dev = "MLP.backward", L._device()
        if self.s is None:
            raise RuntimeError("MLP.backward before MLP.forward")
        self._check_weights(fn, dev)
        _need16(fn, dev, "dy", dy, torch.bfloat16, (self.T, self.K))
        grads = dict(dbias=self.db1, workspace=self.workspace)
        if self.recipe == "fp8_delayed":
            scale, _, amax = self.slots["dy"]
            L.te_quantize_fp8_dbias(dy, E5, self.db2, self.workspace, scale, 0, self.row["dy"], self.col["dy"], amax)
        else:
            L.te_quantize_fp8_dbias(dy, E5, self.db2, self.workspace, self.one)      # the column sums alone
        if self.recipe == "bf16":
            L.te_gemm_bf16(dy, self.h, self.dw2, None, MN, MN)
            L.te_act_bwd_bf16(self.n, self.w1, self.w2, dy, self.z, self.act, self.dz, dx=self.dn, dw=self.dw1, **grads)
        else:
            self._quantize("h", self.h, E4, row=False)
            self._quantize("n", self.n, E4, row=False)
            if self.recipe == "mxfp8":
                self._quantize("dy", dy, E5)
                L.te_act_dgrad_mxfp8(self.row["dy"], self.srow["dy"], self.col["w2"], self.scol["w2"], self.z, self.act,
                                     self.dz, **grads)
            else:
                s = self.slots
                L.te_act_dgrad_fp8(self.row["dy"], E5, self.col["w2"], E4, s["dy"][1], s["w2"][1], self.z, self.act, self.dz,
                                   **grads)
            self._gemm("dy", True, E5, "h", True, E4, self.dw2)
            self._quantize("dz", self.dz, E5)
            self._gemm("dz", False, E5, "w1", True, E4, self.dn)
            self._gemm("dz", True, E5, "n", True, E4, self.dw1)
        L.te_layernorm_bwd(self.dn, self.s, self.gamma, self.mu, self.rsigma, self.dx, self.dgamma, self.dbeta,
                           self.workspace, dres=dy)
        self._end_step()
