"""The norm's and the gated projections' wrappers refuse tensors that are not on the current GPU: another
GPU's addresses would go to a kernel on this one's stream.  Runs on the CPU, with tensors that say which
GPU they are on and a library that only records its calls."""
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from nvfp4_precision_transformer_gb300 import _lib as L

T, K, F, N = 32, 64, 128, 64
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class OnGpu(torch.Tensor):
    is_cuda = True
    index = 0

    def get_device(self):
        return self.index


def gpu(*shape, dtype=BF, index=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    t.index = index
    return t


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name == "te_rmsnorm_bwd_workspace_bytes":
            return lambda rows, cols: rows * cols * 4
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(L, "lib", lambda: rec)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return rec


def one():
    return gpu(1, dtype=F32)


def mx(r, c):
    return gpu(L._mx_bytes(r, c), dtype=U8)


def nv(r, c):
    return gpu(L._nv_bytes(r, c), dtype=U8)


def calls():
    """name -> (function, arguments by name) with every tensor argument given."""
    x, w, h, gu = gpu(T, K), gpu(2 * F, K), gpu(T, F), gpu(T, 2 * F)
    xq, wq, hq = gpu(T, K, dtype=U8), gpu(2 * F, K, dtype=U8), gpu(T, F, dtype=U8)
    norm = dict(x=x, gamma=gpu(K, dtype=F32), eps=1e-5, residual=gpu(T, K), res_out=gpu(T, K), y=gpu(T, K),
                rsigma=gpu(T, dtype=F32), stream=7)
    d = dict(act=0, gu=gu, dgu=gpu(T, 2 * F), stream=7)
    return {
        "rmsnorm_fp8": (te.te_rmsnorm_fp8, dict(norm, fmt=te.E4M3, scale=one(), q_row=xq, amax_out=one(), scale_inv_out=one())),
        "rmsnorm_mxfp8": (te.te_rmsnorm_mxfp8, dict(norm, q_row=xq, s_row=mx(T, K))),
        "rmsnorm_bwd": (te.te_rmsnorm_bwd, dict(dy=x, s=gpu(T, K), gamma=gpu(K, dtype=F32), rsigma=gpu(T, dtype=F32),
                                                dx=gpu(T, K), dgamma=gpu(K, dtype=F32), workspace=gpu(T * K, dtype=F32),
                                                dres=gpu(T, K), stream=7)),
        "gated_bf16": (te.te_gated_gemm_bf16, dict(x=x, w=w, act=0, h=h, gu=gu, stream=7)),
        "gated_fp8": (te.te_gated_gemm_fp8, dict(x=xq, fx=te.E4M3, w=wq, fw=te.E4M3, x_scale_inv=one(), w_scale_inv=one(),
                                                 act=0, h=h, gu=gu, q_h=hq, h_scale=one(), h_amax=one(), h_scale_inv=one(),
                                                 stream=7)),
        "gated_mxfp8": (te.te_gated_gemm_mxfp8, dict(x=xq, sx=mx(T, K), w=wq, sw=mx(2 * F, K), act=0, h=h, gu=gu, q_h=hq,
                                                     s_h=mx(T, F), stream=7)),
        "gated_nvfp4": (te.te_gated_gemm_nvfp4, dict(x=gpu(T, K // 2, dtype=U8), sx=nv(T, K), gx=one(),
                                                     w=gpu(2 * F, K // 2, dtype=U8), sw=nv(2 * F, K), gw=one(), act=0, h=h,
                                                     gu=gu, stream=7)),
        "dgrad_fp8": (te.te_gated_dgrad_fp8, dict(d, dy=gpu(T, N, dtype=U8), fd=te.E5M2, w2=gpu(F, N, dtype=U8), fw=te.E4M3,
                                                  dy_scale_inv=one(), w2_scale_inv=one())),
        "dgrad_mxfp8": (te.te_gated_dgrad_mxfp8, dict(d, dy=gpu(T, N, dtype=U8), sd=mx(T, N), w2=gpu(F, N, dtype=U8),
                                                      sw=mx(F, N))),
        "dgrad_nvfp4": (te.te_gated_dgrad_nvfp4, dict(d, dy=gpu(T, N // 2, dtype=U8), sd=nv(T, N), gd=one(),
                                                      w2=gpu(F, N // 2, dtype=U8), sw=nv(F, N), gw=one())),
        "bwd_bf16": (te.te_gated_bwd_bf16, dict(x=x, w=w, w2=gpu(N, F), dy=gpu(T, N), gu=gu, act=0, dgu=gpu(T, 2 * F),
                                                dx=gpu(T, K), dw=gpu(2 * F, K), stream=7)),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_a_tensor_of_another_gpu_is_refused(library, name):
    fn, args = calls()[name]
    fn(**args)
    assert len(library.calls) == 1
    library.calls.clear()
    for key, value in args.items():
        if isinstance(value, torch.Tensor):
            moved = gpu(*value.shape, dtype=value.dtype, index=1)
            with pytest.raises(ValueError, match=key):
                fn(**{**args, key: moved})
            with pytest.raises(ValueError, match=key):           # on no GPU
                fn(**{**args, key: torch.zeros(*value.shape, dtype=value.dtype)})
    assert library.calls == []


@pytest.mark.parametrize("name", list(calls()))
def test_another_current_device(library, name, monkeypatch):
    """Operands that agree among themselves, but not with the GPU whose stream the call would take."""
    fn, args = calls()[name]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        fn(**args)
    assert library.calls == []
    for value in args.values():
        if isinstance(value, torch.Tensor):
            value.index = 1
    fn(**args)
    assert len(library.calls) == 1


def test_scale_sizes_are_the_librarys():
    """The checks' own arithmetic of scale tensors' sizes, which spares them a call."""
    for rows in (0, 1, 16, 127, 128, 129, 4096):
        for cols in (32, 64, 96, 128, 256, 288, 4096, 4128):
            assert L._mx_bytes(rows, cols) == te.te_scale_bytes(te.E8M0, rows, cols)
            assert L._nv_bytes(rows, cols) == te.te_scale_bytes(te.UE4M3, rows, cols)
