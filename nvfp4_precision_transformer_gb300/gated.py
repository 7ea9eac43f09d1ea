"""The gated feed-forward half of a pre-norm transformer layer as sequences of C-ABI calls.

    r = x + residual
    y = RMSNorm(r) * gamma
    h = act(y Wg^T) * (y Wu^T)        w [2 F, K]: the gate's rows, then the up projection's
    out = h W2^T                      w2 [K, F]

and its backward pass.  Recipes, as in ``linear``:

  bf16         no quantization; any number of tokens in the norm and the gated projections
               (the down projection's GEMMs take multiples of 16)
  fp8_delayed  per-tensor FP8, scales from the amax history (HYBRID: E4M3 y / w / h / w2, E5M2
               gradients); the norm writes y and the gated GEMM writes h in FP8 for the GEMM after it
  mxfp8        1x32 E8M0-scaled E4M3 blocks; likewise (tokens, K, F multiples of 32, F of 128)

Everything here is marshalling: device buffers (torch allocations) and the order of launches;
all arithmetic runs in libte_gb300.so.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .linear import DelayedState

RECIPES = ("bf16", "fp8_delayed", "mxfp8")
FWD_SLOTS = ("y", "w", "h", "w2")
BWD_SLOTS = ("dout", "dgu")
NORM_COLS = 16384       # the most columns that the norms' kernels take


def _need16(fn: str, dev: int, name: str, t, dtype, shape, optional: bool = False) -> None:
    """``L._need``, and the 16-byte boundary that the kernels start from."""
    at = L._need(fn, dev, name, t, dtype, shape, optional)
    if at is not None and at % 16:
        raise ValueError(f"{fn}: {name} does not start on a 16-byte boundary")


class _Block:
    """What the feed-forward blocks share: the quantized copies of their tensors by name, the DelayedScaling state and
    its checkpoint, and the GEMMs on the copies."""

    def _allocate(self, shapes: dict, fwd: tuple, bwd: tuple, history_len: int, dev) -> None:
        """Copies of the tensors (name -> [rows, cols]) and the state of the recipe."""
        u8 = dict(dtype=torch.uint8, device=dev)
        # quantized copies: name -> (row copy, col copy), and for MXFP8 their scales
        if self.recipe != "bf16":
            self.row = {n: torch.empty(r, c, **u8) for n, (r, c) in shapes.items()}
            self.col = {n: torch.empty(c, r, **u8) for n, (r, c) in shapes.items()}
        if self.recipe == "mxfp8":
            self.srow = {n: torch.empty(L.te_scale_bytes(L.E8M0, r, c), **u8) for n, (r, c) in shapes.items()}
            self.scol = {n: torch.empty(L.te_scale_bytes(L.E8M0, c, r), **u8) for n, (r, c) in shapes.items()}
        if self.recipe == "fp8_delayed":
            self.fwd = DelayedState(len(fwd), history_len, dev)
            self.bwd = DelayedState(len(bwd), history_len, dev)
            self.slots = {n: self.fwd.slot(i) for i, n in enumerate(fwd)}
            self.slots.update({n: self.bwd.slot(i) for i, n in enumerate(bwd)})
            self.te_recipe = L.te_recipe(L.E4M3, L.E5M2, history_len, L.ALGO_MAX, 0, 1)
        self.step_idx = 0

    @staticmethod
    def _check_norm(K: int, eps: float) -> None:
        """What the norm, which is not the first launch of a pass, would refuse."""
        if K > NORM_COLS:
            raise ValueError(f"K {K} is more than the {NORM_COLS} columns of the norm")
        if not 0.0 <= eps <= torch.finfo(torch.float32).max:
            raise ValueError(f"eps {eps} is not a finite number >= 0")

    def _end_step(self) -> None:
        """The scales of the next step."""
        if self.recipe == "fp8_delayed":
            for i, st in enumerate((self.fwd, self.bwd)):
                L.te_scale_update(self.te_recipe, i, st.hist, st.amax, st.scale, st.scale_inv, self.step_idx)
        self.step_idx += 1

    def state_dict(self) -> dict:
        """DelayedScaling state of the block (both directions) and its step counter, on the host."""
        if self.recipe != "fp8_delayed":
            return {"step": self.step_idx}
        return {"fwd": self.fwd.state_dict(), "bwd": self.bwd.state_dict(), "step": self.step_idx}

    def load_state_dict(self, sd: dict) -> None:
        if self.recipe == "fp8_delayed":
            self.fwd.load_state_dict(sd["fwd"])
            self.bwd.load_state_dict(sd["bwd"])
        self.step_idx = int(sd["step"])

    # ---- quantization of one tensor under the recipe --------------------------------------------
    def _quantize(self, name: str, t: torch.Tensor, fmt: int, row: bool = True) -> None:
        """Both copies of ``t``; only the col copy where a kernel has written the row copy already."""
        if self.recipe == "mxfp8":
            L.te_quantize_mxfp8(t, self.row[name] if row else None, self.srow[name] if row else None, self.col[name],
                                self.scol[name])
        else:
            scale, _, amax = self.slots[name]
            L.te_quantize_fp8(t, fmt, scale, 0, self.row[name] if row else None, self.col[name], amax if row else None)

    def _gemm(self, a: str, a_col: bool, fa: int, b: str, b_col: bool, fb: int, out: torch.Tensor) -> None:
        """out = A B^T from the named copies."""
        A, B = (self.col if a_col else self.row)[a], (self.col if b_col else self.row)[b]
        if self.recipe == "mxfp8":
            L.te_gemm_mxfp8(A, (self.scol if a_col else self.srow)[a], B, (self.scol if b_col else self.srow)[b], out)
        else:
            L.te_gemm_fp8(A, fa, B, fb, self.slots[a][1], self.slots[b][1], out)


class GatedMLP(_Block):
    """Device buffers of one gated feed-forward block for ``tokens`` tokens, its forward and backward pass.

    ``forward(x, residual)`` returns (out, r): the block's output and the next residual, whose sum is
    the next block's input.  ``backward(dout, dr)`` takes their gradients (dr may be None) and leaves
    ``dx`` (the gradient of x and of residual alike), ``dgamma``, ``dw`` and ``dw2``.

    x, residual (or None) and dr are contiguous bf16 [tokens, K], K at most 16384; w, w2 and dout too, or fp32 where
    the recipe quantizes them; all on 16-byte boundaries.  Anything else is refused before the first launch."""

    def __init__(self, gamma: torch.Tensor, w: torch.Tensor, w2: torch.Tensor, tokens: int, recipe: str = "bf16",
                 act: int = L.ACT_SILU, eps: float = 1e-5, history_len: int = 16):
        if recipe not in RECIPES:
            raise ValueError(f"recipe {recipe!r} is none of {RECIPES}")
        F2, K = w.shape
        F = F2 // 2
        if w2.shape != (K, F) or gamma.shape != (K,):
            raise ValueError(f"gamma {tuple(gamma.shape)}, w {tuple(w.shape)} and w2 {tuple(w2.shape)} are not "
                             "[K], [2 F, K] and [K, F]")
        self.gamma, self.w, self.w2 = gamma, w, w2
        self.T, self.K, self.F, self.recipe, self.act, self.eps = tokens, K, F, recipe, act, eps
        self._check_norm(K, eps)
        self._check_weights("GatedMLP", L._device())
        dev, T = w.device, tokens
        bf, f32 = (dict(dtype=t, device=dev) for t in (torch.bfloat16, torch.float32))
        self.r, self.y, self.h = torch.empty(T, K, **bf), torch.empty(T, K, **bf), torch.empty(T, F, **bf)
        self.gu, self.dgu = torch.empty(T, 2 * F, **bf), torch.empty(T, 2 * F, **bf)
        self.out, self.dy, self.dx = (torch.empty(T, K, **bf) for _ in range(3))
        self.dw, self.dw2 = torch.empty(2 * F, K, **bf), torch.empty(K, F, **bf)
        self.rsigma, self.dgamma = torch.empty(T, **f32), torch.empty(K, **f32)
        self.workspace = torch.empty(L.te_rmsnorm_bwd_workspace_bytes(T, K) // 4, **f32)
        self._allocate({"y": (T, K), "w": (2 * F, K), "h": (T, F), "w2": (K, F), "dout": (T, K), "dgu": (T, 2 * F)},
                       FWD_SLOTS, BWD_SLOTS, history_len, dev)

    # ---- checks: before the first launch of a pass, whose calls take addresses and sizes as they are ----
    def _operand(self, fn: str, dev: int, name: str, t: torch.Tensor, shape: tuple) -> None:
        """A tensor that the BF16 GEMMs or the quantizers (which take fp32 too) read."""
        _need16(fn, dev, name, t, torch.bfloat16 if self.recipe == "bf16" else (torch.bfloat16, torch.float32), shape)

    def _check_weights(self, fn: str, dev: int) -> None:
        _need16(fn, dev, "gamma", self.gamma, torch.float32, (self.K,))
        self._operand(fn, dev, "w", self.w, (2 * self.F, self.K))
        self._operand(fn, dev, "w2", self.w2, (self.K, self.F))

    # ---- passes ----------------------------------------------------------------------------------
    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        E4, tokens = L.E4M3, (self.T, self.K)
        fn, dev = "GatedMLP.forward", L._device()
        self._check_weights(fn, dev)
        _need16(fn, dev, "x", x, torch.bfloat16, tokens)
        _need16(fn, dev, "residual", residual, torch.bfloat16, tokens, True)
        if self.recipe == "bf16":
            L.te_rmsnorm_fp8(x, self.gamma, self.eps, E4, residual=residual, res_out=self.r, y=self.y, rsigma=self.rsigma)
            L.te_gated_gemm_bf16(self.y, self.w, self.act, h=self.h, gu=self.gu)
            L.te_gemm_bf16(self.h, self.w2, self.out)
            return self.out, self.r
        self._quantize("w", self.w, E4)
        self._quantize("w2", self.w2, E4)
        if self.recipe == "mxfp8":
            L.te_rmsnorm_mxfp8(x, self.gamma, self.eps, self.row["y"], self.srow["y"], residual=residual, res_out=self.r,
                               y=self.y, rsigma=self.rsigma)
            L.te_gated_gemm_mxfp8(self.row["y"], self.srow["y"], self.row["w"], self.srow["w"], self.act, h=self.h,
                                  gu=self.gu, q_h=self.row["h"], s_h=self.srow["h"])
        else:
            s = self.slots
            L.te_rmsnorm_fp8(x, self.gamma, self.eps, E4, s["y"][0], self.row["y"], residual=residual, res_out=self.r,
                             y=self.y, rsigma=self.rsigma, amax_out=s["y"][2])
            L.te_gated_gemm_fp8(self.row["y"], E4, self.row["w"], E4, s["y"][1], s["w"][1], self.act, h=self.h, gu=self.gu,
                                q_h=self.row["h"], h_fmt=E4, h_scale=s["h"][0], h_amax=s["h"][2])
        self._gemm("h", False, E4, "w2", False, E4, self.out)
        return self.out, self.r

    def backward(self, dout: torch.Tensor, dr: torch.Tensor | None = None) -> None:
        E4, E5, MN = L.E4M3, L.E5M2, L.MN_MAJOR
        fn, dev = "GatedMLP.backward", L._device()
        self._check_weights(fn, dev)
        self._operand(fn, dev, "dout", dout, (self.T, self.K))
        _need16(fn, dev, "dr", dr, torch.bfloat16, (self.T, self.K), True)
        if self.recipe == "bf16":
            L.te_gemm_bf16(dout, self.h, self.dw2, None, MN, MN)
            L.te_gated_bwd_bf16(self.y, self.w, self.w2, dout, self.gu, self.act, self.dgu, dx=self.dy, dw=self.dw)
        else:
            self._quantize("dout", dout, E5)
            self._quantize("h", self.h, E4, row=False)
            self._quantize("y", self.y, E4, row=False)
            self._gemm("dout", True, E5, "h", True, E4, self.dw2)
            if self.recipe == "mxfp8":
                L.te_gated_dgrad_mxfp8(self.row["dout"], self.srow["dout"], self.col["w2"], self.scol["w2"], self.gu,
                                       self.act, self.dgu)
            else:
                s = self.slots
                L.te_gated_dgrad_fp8(self.row["dout"], E5, self.col["w2"], E4, s["dout"][1], s["w2"][1], self.gu, self.act,
                                     self.dgu)
            self._quantize("dgu", self.dgu, E5)
            self._gemm("dgu", False, E5, "w", True, E4, self.dy)
            self._gemm("dgu", True, E5, "y", True, E4, self.dw)
        L.te_rmsnorm_bwd(self.dy, self.r, self.gamma, self.rsigma, self.dx, self.dgamma, self.workspace, dres=dr)
        self._end_step()
