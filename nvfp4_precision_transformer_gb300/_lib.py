"""ctypes binding of libte_gb300.so (argument marshalling only).

Every function here has the name of the C entry point it wraps and does no
arithmetic of its own: it turns torch tensors into device pointers and sizes,
passes the current CUDA stream, and raises TEError on a non-zero status.  The
library must have been built (``build.build()``); importing this module fails
loudly otherwise -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libte_gb300.so")

# te_dtype
F32, BF16, E4M3, E5M2, E2M1, E8M0, UE4M3 = range(7)
# NVFP4 flags
NVFP4_2D, NVFP4_RHT_COL, NVFP4_SR = 1, 2, 4
ALGO_MAX, ALGO_MOST_RECENT = 0, 1
# gated activations
ACT_SILU, ACT_GELU = 0, 1
# te_layout
K_MAJOR, MN_MAJOR = 0, 1

STATUS = {0: "TE_OK", 1: "TE_ERR_NULL", 2: "TE_ERR_SHAPE", 3: "TE_ERR_ALIGN", 4: "TE_ERR_DTYPE",
          5: "TE_ERR_UNSUPPORTED", 6: "TE_ERR_CUDA", 7: "TE_ERR_TIMEOUT", 8: "TE_ERR_ARG"}

# exported symbols and their signatures (restype, argtypes)
_vp, _i64, _u32, _u64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int
_st = ctypes.c_int


class te_recipe(ctypes.Structure):
    _fields_ = [("fwd_fmt", ctypes.c_int), ("bwd_fmt", ctypes.c_int), ("amax_history_len", ctypes.c_int),
                ("amax_compute_algo", ctypes.c_int), ("margin", ctypes.c_int), ("interval", ctypes.c_int)]


SIGNATURES = {
    "te_amax_reduce": (_st, [_vp, _int, _i64, _i64, _vp, _vp, _u32, _vp]),
    "te_scale_update": (_st, [ctypes.POINTER(te_recipe), _int, _int, _vp, _vp, _vp, _vp, _i64, _vp]),
    "te_quantize_fp8": (_st, [_vp, _int, _i64, _i64, _int, _vp, _int, _vp, _vp, _vp, _vp, _vp]),
    "te_quantize_mxfp8": (_st, [_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "te_layernorm_fp8": (_st, [_vp, _int, _i64, _i64, _vp, _vp, ctypes.c_float, _int, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _vp]),
    "te_quantize_fp8_dbias_noalloc": (_st, [_vp, _int, _i64, _i64, _int, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "te_dbias_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "te_quantize_fp8_dbias": (_st, [_vp, _int, _i64, _i64, _int, _vp, _int, _vp, _vp, _vp, _vp, _vp, _vp,
                                    ctypes.c_size_t, _vp]),
    "te_rmsnorm_fp8": (_st, [_vp, _int, _i64, _i64, _vp, _vp, ctypes.c_float, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                             _vp]),
    "te_rmsnorm_mxfp8": (_st, [_vp, _int, _i64, _i64, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp]),
    "te_rmsnorm_bwd_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "te_rmsnorm_bwd": (_st, [_vp, _vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "te_quantize_nvfp4": (_st, [_vp, _int, _i64, _i64, _u32, _u32, _u64, _u64, _vp, _vp,
                                _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "te_gemm_bf16": (_st, [_vp, _int, _vp, _int, _vp, _vp, _int, _int, _i64, _i64, _i64, _vp]),
    "te_gemm_fp8": (_st, [_vp, _int, _vp, _int, _vp, _vp, _vp, _vp, _int, _int, _i64, _i64, _i64, _vp]),
    "te_gemm_mxfp8": (_st, [_vp, _int, _vp, _vp, _int, _vp, _vp, _vp, _int, _int, _i64, _i64, _i64, _vp]),
    "te_gemm_nvfp4": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _i64, _i64, _i64, _vp]),
    "te_gated_gemm_bf16": (_st, [_vp, _vp, _int, _vp, _vp, _i64, _i64, _i64, _vp]),
    "te_gated_gemm_fp8": (_st, [_vp, _int, _vp, _int, _vp, _vp, _int, _vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _i64,
                                _i64, _vp]),
    "te_gated_gemm_mxfp8": (_st, [_vp, _int, _vp, _vp, _int, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "te_gated_gemm_nvfp4": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _i64, _i64, _i64, _vp]),
    "te_gated_dgrad_fp8": (_st, [_vp, _int, _vp, _int, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64, _vp]),
    "te_gated_dgrad_mxfp8": (_st, [_vp, _int, _vp, _vp, _int, _vp, _vp, _int, _vp, _i64, _i64, _i64, _vp]),
    "te_gated_dgrad_nvfp4": (_st, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _i64, _i64, _i64, _vp]),
    "te_gated_bwd_bf16": (_st, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _int, _int, _i64, _i64, _i64, _i64,
                                _vp]),
    "te_scale_bytes": (ctypes.c_size_t, [_int, _i64, _i64]),
    "te_scale_unswizzle": (_st, [_int, _i64, _i64, _vp, _vp]),
    "te_status_str": (ctypes.c_char_p, [_int]),
    "te_get_last_error": (_st, []),
    "te_launch_count": (_u64, []),
    "te_selftest_wait_timeout": (_st, [_vp]),
}


class TEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with nvfp4_precision_transformer_gb300.build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


def _check(name: str, status: int) -> None:
    if status != 0:
        raise TEError(name, status)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_bf16, _f32, _u8 = torch.bfloat16, torch.float32, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev=None):
    if stream is None:
        # the handle alone: building a Stream object takes 3 us, as long as a small kernel
        dev = torch.cuda.current_device() if dev is None else dev
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _in_dtype(x):
    if x.dtype == torch.bfloat16:
        return BF16
    if x.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported input dtype {x.dtype}")


def _rc(x):
    assert x.dim() == 2 and x.is_contiguous()
    return x.shape[0], x.shape[1]


# ---- entry points (same names as the C ABI) ----------------------------------------

def te_amax_reduce(x, amax, amax_rht=None, rht_signs: int = 0, stream=None):
    r, c = _rc(x)
    _check("te_amax_reduce", lib().te_amax_reduce(_ptr(x), _in_dtype(x), r, c, _ptr(amax), _ptr(amax_rht),
                                                  rht_signs & 0xFFFFFFFF, _stream(stream)))


def te_scale_update(recipe: te_recipe, is_backward: int, hist, amax, scale, scale_inv, step: int, stream=None):
    n = amax.numel()
    _check("te_scale_update", lib().te_scale_update(ctypes.byref(recipe), int(is_backward), n, _ptr(hist),
                                                    _ptr(amax), _ptr(scale), _ptr(scale_inv), int(step),
                                                    _stream(stream)))


def te_quantize_fp8(x, fmt: int, scale=None, compute_scale: int = 0, q_row=None, q_col=None, amax_out=None,
                    scale_inv_out=None, stream=None):
    r, c = _rc(x)
    _check("te_quantize_fp8", lib().te_quantize_fp8(_ptr(x), _in_dtype(x), r, c, fmt, _ptr(scale), compute_scale,
                                                    _ptr(q_row), _ptr(q_col), _ptr(amax_out), _ptr(scale_inv_out),
                                                    _stream(stream)))


def te_dbias_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().te_dbias_workspace_bytes(rows, cols))


def te_quantize_fp8_dbias(x, fmt: int, dbias, workspace, scale=None, compute_scale: int = 0, q_row=None, q_col=None,
                          amax_out=None, scale_inv_out=None, stream=None):
    r, c = _rc(x)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("te_quantize_fp8_dbias", lib().te_quantize_fp8_dbias(
        _ptr(x), _in_dtype(x), r, c, fmt, _ptr(scale), compute_scale, _ptr(q_row), _ptr(q_col), _ptr(amax_out),
        _ptr(scale_inv_out), _ptr(dbias), _ptr(workspace), nbytes, _stream(stream)))


def te_quantize_fp8_dbias_noalloc(x, fmt: int, dbias, scale=None, compute_scale: int = 0, q_row=None, q_col=None,
                                  amax_out=None, scale_inv_out=None, stream=None):
    """te_quantize_fp8_dbias with the library's fixed scratch array instead of a workspace."""
    r, c = _rc(x)
    _check("te_quantize_fp8_dbias_noalloc", lib().te_quantize_fp8_dbias_noalloc(
        _ptr(x), _in_dtype(x), r, c, fmt, _ptr(scale), compute_scale, _ptr(q_row), _ptr(q_col), _ptr(amax_out),
        _ptr(scale_inv_out), _ptr(dbias), _stream(stream)))


def te_layernorm_fp8(x, gamma, beta, eps: float, fmt: int, scale, q_row, ln_out=None, mu=None, rsigma=None,
                     amax_out=None, scale_inv_out=None, stream=None):
    r, c = _rc(x)
    _check("te_layernorm_fp8", lib().te_layernorm_fp8(
        _ptr(x), _in_dtype(x), r, c, _ptr(gamma), _ptr(beta), float(eps), fmt, _ptr(scale), _ptr(q_row),
        _ptr(ln_out), _ptr(mu), _ptr(rsigma), _ptr(amax_out), _ptr(scale_inv_out), _stream(stream)))


def _device() -> int:
    """The current GPU, whose stream a call goes to; -2, where no tensor is, without one."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


def _misplaced(fn: str, dev: int, name: str, t) -> ValueError:
    if not t.is_cuda or dev < 0:
        return ValueError(f"{fn}: {name} is not on the GPU")
    return ValueError(f"{fn}: {name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")


def _need(fn: str, dev: int, name: str, t, dtype, shape, optional: bool = False):
    """Refuses a tensor that the call would misread: not on GPU ``dev``, not contiguous, of another
    dtype (one, or a tuple of them) or shape.  Returns its address."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{fn}: {name} is required")
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{fn}: {name} is {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} is not contiguous")
    if t.get_device() != dev:
        raise _misplaced(fn, dev, name, t)
    return t.data_ptr()


def _need_n(fn: str, dev: int, name: str, t, dtype, n: int, optional: bool = False):
    """The same for a tensor of at least ``n`` elements whatever its shape (scalars, scale tensors)."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{fn}: {name} is required")
    if t.dtype is dtype and t.numel() >= n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{fn}: {name} is {t.dtype}, expected {dtype}")
    if t.numel() < n:
        raise ValueError(f"{fn}: {name} has {t.numel()} elements, needs {n}")
    if t.get_device() != dev:
        raise _misplaced(fn, dev, name, t)
    raise ValueError(f"{fn}: {name} is not contiguous")


def _mx_bytes(rows: int, cols: int) -> int:
    """te_scale_bytes(E8M0, rows, cols) of whole blocks."""
    return -(-rows // 128) * 128 * (-(-cols // 128) * 4)


def _nv_bytes(rows: int, cols: int) -> int:
    """te_scale_bytes(UE4M3, rows, cols) of whole blocks."""
    return -(-rows // 128) * 128 * (-(-cols // 256) * 16)


def _norm_operands(fn, dev, x, gamma, residual, res_out, y, rsigma):
    if x.dim() != 2:
        raise ValueError(f"{fn}: x has shape {tuple(x.shape)}, expected [rows, cols]")
    shape, dt = x.shape, x.dtype
    rows, cols = shape
    px = _need(fn, dev, "x", x, dt if dt is _bf16 or dt is _f32 else (_bf16, _f32), shape)
    return (px, F32 if dt is _f32 else BF16, rows, cols, _need(fn, dev, "residual", residual, dt, shape, True),
            _need(fn, dev, "gamma", gamma, _f32, (cols,)), _need(fn, dev, "res_out", res_out, dt, shape, True),
            _need(fn, dev, "y", y, _bf16, shape, True), _need(fn, dev, "rsigma", rsigma, _f32, (rows,), True))


def te_rmsnorm_fp8(x, gamma, eps: float, fmt: int, scale=None, q_row=None, residual=None, res_out=None, y=None,
                   rsigma=None, amax_out=None, scale_inv_out=None, stream=None):
    """RMSNorm of x (+ residual), its output in FP8 with a per-tensor scale (and / or y in bf16)."""
    fn = "te_rmsnorm_fp8"
    dev = _device()
    px, dt, r, c, pres, pg, pro, py, prs = _norm_operands(fn, dev, x, gamma, residual, res_out, y, rsigma)
    _check(fn, lib().te_rmsnorm_fp8(
        px, dt, r, c, pres, pg, float(eps), fmt, _need_n(fn, dev, "scale", scale, _f32, 1, True),
        _need(fn, dev, "q_row", q_row, _u8, x.shape, True), py, pro, prs,
        _need_n(fn, dev, "amax_out", amax_out, _f32, 1, True),
        _need_n(fn, dev, "scale_inv_out", scale_inv_out, _f32, 1, True),
        _stream(stream, dev)))


def te_rmsnorm_mxfp8(x, gamma, eps: float, q_row, s_row, residual=None, res_out=None, y=None, rsigma=None, stream=None):
    """RMSNorm of x (+ residual), its output in MXFP8 (E4M3 codes, E8M0 scales in the tensor-core layout)."""
    fn = "te_rmsnorm_mxfp8"
    dev = _device()
    px, dt, r, c, pres, pg, pro, py, prs = _norm_operands(fn, dev, x, gamma, residual, res_out, y, rsigma)
    _check(fn, lib().te_rmsnorm_mxfp8(
        px, dt, r, c, pres, pg, float(eps), _need(fn, dev, "q_row", q_row, _u8, x.shape),
        _need_n(fn, dev, "s_row", s_row, _u8, _mx_bytes(r, c)), py, pro, prs, _stream(stream, dev)))


def te_rmsnorm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().te_rmsnorm_bwd_workspace_bytes(rows, cols))


def te_rmsnorm_bwd(dy, s, gamma, rsigma, dx, dgamma, workspace, dres=None, stream=None):
    """Gradients of te_rmsnorm_*: dx (of x and of the residual) and dgamma."""
    fn = "te_rmsnorm_bwd"
    dev = _device()
    if s.dim() != 2:
        raise ValueError(f"{fn}: s has shape {tuple(s.shape)}, expected [rows, cols]")
    shape, dt = s.shape, s.dtype
    ps = _need(fn, dev, "s", s, (_bf16, _f32), shape)
    pw = _need_n(fn, dev, "workspace", workspace, _f32, 0)
    _check(fn, lib().te_rmsnorm_bwd(
        _need(fn, dev, "dy", dy, _bf16, shape), ps, _in_dtype(s), shape[0], shape[1],
        _need(fn, dev, "gamma", gamma, _f32, shape[1:]), _need(fn, dev, "rsigma", rsigma, _f32, shape[:1]),
        _need(fn, dev, "dres", dres, dt, shape, True), _need(fn, dev, "dx", dx, dt, shape),
        _need(fn, dev, "dgamma", dgamma, _f32, shape[1:]), pw, workspace.numel() * 4, _stream(stream, dev)))


def te_quantize_mxfp8(x, q_row=None, s_row=None, q_col=None, s_col=None, stream=None):
    r, c = _rc(x)
    _check("te_quantize_mxfp8", lib().te_quantize_mxfp8(_ptr(x), _in_dtype(x), r, c, _ptr(q_row), _ptr(s_row),
                                                        _ptr(q_col), _ptr(s_col), _stream(stream)))


def te_quantize_nvfp4(x, flags: int = 0, rht_signs: int = 0, seed: int = 0, offset: int = 0, amax=None,
                      amax_rht=None, q_row=None, s_row=None, gdec_row=None, q_col=None, s_col=None, gdec_col=None,
                      stream=None):
    r, c = _rc(x)
    _check("te_quantize_nvfp4", lib().te_quantize_nvfp4(_ptr(x), _in_dtype(x), r, c, flags, rht_signs, seed,
                                                        offset, _ptr(amax), _ptr(amax_rht), _ptr(q_row),
                                                        _ptr(s_row), _ptr(gdec_row), _ptr(q_col), _ptr(s_col),
                                                        _ptr(gdec_col), _stream(stream)))


def _out_dtype(d):
    if d.dtype == torch.bfloat16:
        return BF16
    if d.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported output dtype {d.dtype}")


# accumulate=1: D (fp32) += the GEMM's result instead of D = result (Wgrad into a main
# gradient); the library rejects it for a bf16 D.

def te_gemm_bf16(A, B, D, bias=None, a_layout: int = 0, b_layout: int = 0, accumulate: int = 0, stream=None):
    """A is [M, K] (K_MAJOR) or [K, M] (MN_MAJOR); B is [N, K] or [K, N]; D is [M, N]."""
    M, N = D.shape
    K = A.shape[1] if a_layout == K_MAJOR else A.shape[0]
    _check("te_gemm_bf16", lib().te_gemm_bf16(_ptr(A), a_layout, _ptr(B), b_layout, _ptr(bias), _ptr(D),
                                              _out_dtype(D), int(accumulate), M, N, K, _stream(stream)))


def te_gemm_fp8(A, fa: int, B, fb: int, a_scale_inv, b_scale_inv, D, bias=None, accumulate: int = 0, stream=None):
    M, K = A.shape
    N = B.shape[0]
    _check("te_gemm_fp8", lib().te_gemm_fp8(_ptr(A), fa, _ptr(B), fb, _ptr(a_scale_inv), _ptr(b_scale_inv),
                                            _ptr(bias), _ptr(D), _out_dtype(D), int(accumulate), M, N, K,
                                            _stream(stream)))


def te_gemm_mxfp8(A, sA, B, sB, D, bias=None, fa: int = E4M3, fb: int = E4M3, accumulate: int = 0, stream=None):
    M, K = A.shape
    N = B.shape[0]
    _check("te_gemm_mxfp8", lib().te_gemm_mxfp8(_ptr(A), fa, _ptr(sA), _ptr(B), fb, _ptr(sB), _ptr(bias), _ptr(D),
                                                _out_dtype(D), int(accumulate), M, N, K, _stream(stream)))


def te_gemm_nvfp4(A, sA, gA, B, sB, gB, D, bias=None, accumulate: int = 0, stream=None):
    M, Kh = A.shape
    N = B.shape[0]
    _check("te_gemm_nvfp4", lib().te_gemm_nvfp4(_ptr(A), _ptr(sA), _ptr(gA), _ptr(B), _ptr(sB), _ptr(gB),
                                                _ptr(bias), _ptr(D), _out_dtype(D), int(accumulate), M, N, 2 * Kh,
                                                _stream(stream)))


# ---- gated feed-forward projections: w [2 F, K] holds the gate's rows, then the up projection's --------

def _gated_shape(fn, x, w, packed: int = 1):
    """(T, K, F) of x [T, K / packed] and w [2 F, K / packed]."""
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1] or w.shape[0] % 2:
        raise ValueError(f"{fn}: x {tuple(x.shape)} and w {tuple(w.shape)} are not [T, K] and [2 F, K]")
    return x.shape[0], x.shape[1] * packed, w.shape[0] // 2


def te_gated_gemm_bf16(x, w, act: int, h=None, gu=None, stream=None):
    """h = act(x Wg^T) * (x Wu^T) in bf16 and / or the pre-activations gu = [g, u]."""
    fn = "te_gated_gemm_bf16"
    dev = _device()
    T, K, F = _gated_shape(fn, x, w)
    _check(fn, lib().te_gated_gemm_bf16(
        _need(fn, dev, "x", x, _bf16, (T, K)), _need(fn, dev, "w", w, _bf16, (2 * F, K)), act,
        _need(fn, dev, "h", h, _bf16, (T, F), True), _need(fn, dev, "gu", gu, _bf16, (T, 2 * F), True), T, K, F,
        _stream(stream, dev)))


def te_gated_gemm_fp8(x, fx: int, w, fw: int, x_scale_inv, w_scale_inv, act: int, h=None, gu=None, q_h=None,
                      h_fmt: int = E4M3, h_scale=None, h_amax=None, h_scale_inv=None, stream=None):
    """te_gated_gemm_bf16 on per-tensor scaled FP8 operands; q_h is h in FP8 for the down projection."""
    fn = "te_gated_gemm_fp8"
    dev = _device()
    T, K, F = _gated_shape(fn, x, w)
    _check(fn, lib().te_gated_gemm_fp8(
        _need(fn, dev, "x", x, _u8, (T, K)), fx, _need(fn, dev, "w", w, _u8, (2 * F, K)), fw,
        _need_n(fn, dev, "x_scale_inv", x_scale_inv, _f32, 1), _need_n(fn, dev, "w_scale_inv", w_scale_inv, _f32, 1), act,
        _need(fn, dev, "h", h, _bf16, (T, F), True), _need(fn, dev, "gu", gu, _bf16, (T, 2 * F), True),
        _need(fn, dev, "q_h", q_h, _u8, (T, F), True), h_fmt, _need_n(fn, dev, "h_scale", h_scale, _f32, 1, True),
        _need_n(fn, dev, "h_amax", h_amax, _f32, 1, True), _need_n(fn, dev, "h_scale_inv", h_scale_inv, _f32, 1, True),
        T, K, F, _stream(stream, dev)))


def te_gated_gemm_mxfp8(x, sx, w, sw, act: int, h=None, gu=None, q_h=None, s_h=None, fx: int = E4M3, fw: int = E4M3,
                        stream=None):
    """te_gated_gemm_bf16 on MXFP8 operands; q_h, s_h are h in MXFP8 for the down projection."""
    fn = "te_gated_gemm_mxfp8"
    dev = _device()
    T, K, F = _gated_shape(fn, x, w)
    _check(fn, lib().te_gated_gemm_mxfp8(
        _need(fn, dev, "x", x, _u8, (T, K)), fx, _need_n(fn, dev, "sx", sx, _u8, _mx_bytes(T, K)),
        _need(fn, dev, "w", w, _u8, (2 * F, K)), fw, _need_n(fn, dev, "sw", sw, _u8, _mx_bytes(2 * F, K)), act,
        _need(fn, dev, "h", h, _bf16, (T, F), True), _need(fn, dev, "gu", gu, _bf16, (T, 2 * F), True),
        _need(fn, dev, "q_h", q_h, _u8, (T, F), True), _need_n(fn, dev, "s_h", s_h, _u8, _mx_bytes(T, F), True), T, K, F,
        _stream(stream, dev)))


def te_gated_gemm_nvfp4(x, sx, gx, w, sw, gw, act: int, h=None, gu=None, stream=None):
    """te_gated_gemm_bf16 on NVFP4 operands (packed codes, block scales, tensor scales)."""
    fn = "te_gated_gemm_nvfp4"
    dev = _device()
    T, K, F = _gated_shape(fn, x, w, 2)
    _check(fn, lib().te_gated_gemm_nvfp4(
        _need(fn, dev, "x", x, _u8, (T, K // 2)), _need_n(fn, dev, "sx", sx, _u8, _nv_bytes(T, K)),
        _need_n(fn, dev, "gx", gx, _f32, 1), _need(fn, dev, "w", w, _u8, (2 * F, K // 2)),
        _need_n(fn, dev, "sw", sw, _u8, _nv_bytes(2 * F, K)), _need_n(fn, dev, "gw", gw, _f32, 1), act,
        _need(fn, dev, "h", h, _bf16, (T, F), True), _need(fn, dev, "gu", gu, _bf16, (T, 2 * F), True), T, K, F,
        _stream(stream, dev)))


def _dgrad_shape(fn, dev, dy, w2, gu, dgu, packed: int = 1):
    """(T, F, N) of dy [T, N / packed] and W2's col copy [F, N / packed], and the pointers of gu and dgu."""
    if dy.dim() != 2 or w2.dim() != 2 or dy.shape[1] != w2.shape[1]:
        raise ValueError(f"{fn}: dy {tuple(dy.shape)} and w2 {tuple(w2.shape)} are not [T, N] and [F, N]")
    T, F = dy.shape[0], w2.shape[0]
    return (T, F, dy.shape[1] * packed, _need(fn, dev, "gu", gu, _bf16, (T, 2 * F)),
            _need(fn, dev, "dgu", dgu, _bf16, (T, 2 * F)))


def te_gated_dgrad_fp8(dy, fd: int, w2, fw: int, dy_scale_inv, w2_scale_inv, gu, act: int, dgu, stream=None):
    """Gradients of the pre-activations from dy's row copy [T, N] and W2's col copy [F, N] in FP8."""
    fn = "te_gated_dgrad_fp8"
    dev = _device()
    T, F, N, pgu, pdgu = _dgrad_shape(fn, dev, dy, w2, gu, dgu)
    _check(fn, lib().te_gated_dgrad_fp8(
        _need(fn, dev, "dy", dy, _u8, (T, N)), fd, _need(fn, dev, "w2", w2, _u8, (F, N)), fw,
        _need_n(fn, dev, "dy_scale_inv", dy_scale_inv, _f32, 1), _need_n(fn, dev, "w2_scale_inv", w2_scale_inv, _f32, 1), pgu,
        act, pdgu, T, F, N, _stream(stream, dev)))


def te_gated_dgrad_mxfp8(dy, sd, w2, sw, gu, act: int, dgu, fd: int = E4M3, fw: int = E4M3, stream=None):
    """te_gated_dgrad_fp8 on MXFP8 copies."""
    fn = "te_gated_dgrad_mxfp8"
    dev = _device()
    T, F, N, pgu, pdgu = _dgrad_shape(fn, dev, dy, w2, gu, dgu)
    _check(fn, lib().te_gated_dgrad_mxfp8(
        _need(fn, dev, "dy", dy, _u8, (T, N)), fd, _need_n(fn, dev, "sd", sd, _u8, _mx_bytes(T, N)),
        _need(fn, dev, "w2", w2, _u8, (F, N)), fw, _need_n(fn, dev, "sw", sw, _u8, _mx_bytes(F, N)), pgu, act, pdgu, T, F, N,
        _stream(stream, dev)))


def te_gated_dgrad_nvfp4(dy, sd, gd, w2, sw, gw, gu, act: int, dgu, stream=None):
    """te_gated_dgrad_fp8 on NVFP4 copies."""
    fn = "te_gated_dgrad_nvfp4"
    dev = _device()
    T, F, N, pgu, pdgu = _dgrad_shape(fn, dev, dy, w2, gu, dgu, 2)
    _check(fn, lib().te_gated_dgrad_nvfp4(
        _need(fn, dev, "dy", dy, _u8, (T, N // 2)), _need_n(fn, dev, "sd", sd, _u8, _nv_bytes(T, N)),
        _need_n(fn, dev, "gd", gd, _f32, 1), _need(fn, dev, "w2", w2, _u8, (F, N // 2)),
        _need_n(fn, dev, "sw", sw, _u8, _nv_bytes(F, N)), _need_n(fn, dev, "gw", gw, _f32, 1), pgu, act, pdgu, T, F, N,
        _stream(stream, dev)))


def te_gated_bwd_bf16(x, w, w2, dy, gu, act: int, dgu, dx=None, dw=None, accumulate: int = 0, stream=None):
    """The BF16 backward pass: dgu from dy [T, N] and w2 [N, F], then dx = dgu w and dw (+)= dgu^T x."""
    fn = "te_gated_bwd_bf16"
    dev = _device()
    T, K, F = _gated_shape(fn, x, w)
    if dy.dim() != 2:
        raise ValueError(f"{fn}: dy has shape {tuple(dy.shape)}, expected [T, N]")
    N = dy.shape[1]
    _check(fn, lib().te_gated_bwd_bf16(
        _need(fn, dev, "x", x, _bf16, (T, K)), _need(fn, dev, "w", w, _bf16, (2 * F, K)), _need(fn, dev, "w2", w2, _bf16, (N, F)),
        _need(fn, dev, "dy", dy, _bf16, (T, N)), _need(fn, dev, "gu", gu, _bf16, (T, 2 * F)), act,
        _need(fn, dev, "dgu", dgu, _bf16, (T, 2 * F)), _need(fn, dev, "dx", dx, _bf16, (T, K), True),
        _need(fn, dev, "dw", dw, (_bf16, _f32), (2 * F, K), True), BF16 if dw is None else _out_dtype(dw),
        int(accumulate), T, K, F, N, _stream(stream, dev)))


def te_scale_bytes(scale_fmt: int, rows: int, cols: int) -> int:
    return int(lib().te_scale_bytes(scale_fmt, rows, cols))


def te_scale_unswizzle(scale_fmt: int, rows: int, cols: int, swizzled: np.ndarray) -> np.ndarray:
    blk = 32 if scale_fmt == E8M0 else 16
    sw = np.ascontiguousarray(swizzled, dtype=np.uint8)
    out = np.zeros((rows, cols // blk), dtype=np.uint8)
    _check("te_scale_unswizzle", lib().te_scale_unswizzle(scale_fmt, rows, cols, sw.ctypes.data,
                                                          out.ctypes.data))
    return out


def te_status_str(status: int) -> str:
    return lib().te_status_str(status).decode()


def te_get_last_error() -> int:
    return int(lib().te_get_last_error())


def te_launch_count() -> int:
    return int(lib().te_launch_count())


def te_selftest_wait_timeout(stream=None):
    _check("te_selftest_wait_timeout", lib().te_selftest_wait_timeout(_stream(stream)))
