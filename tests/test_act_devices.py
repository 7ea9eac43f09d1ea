"""The wrappers of LayerNorm and of the linear with bias, activation and residual refuse tensors that are not on the
current GPU, by name, before the library is called.  Runs on the CPU, as test_wrapper_devices."""
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests.test_wrapper_devices import F32, U8, Recorder, gpu, library, mx, nv, one  # noqa: F401

T, K, N = 32, 64, 128


def calls():
    """name -> (function, arguments by name) with every tensor argument given."""
    v = lambda n: gpu(n, dtype=F32)   # noqa: E731
    q = lambda *s: gpu(*s, dtype=U8)   # noqa: E731
    norm = dict(x=gpu(T, K), gamma=v(K), beta=v(K), eps=1e-5, residual=gpu(T, K), res_out=gpu(T, K), y=gpu(T, K), mu=v(T),
                rsigma=v(T), stream=7)
    out = dict(act=te.ACT_GELU, y=gpu(T, N), z=gpu(T, N), bias=v(N), stream=7)
    res = dict(out, residual=gpu(T, N))
    grad = dict(z=gpu(T, N), act=te.ACT_GELU, dz=gpu(T, N), dbias=v(N), workspace=v(N), stream=7)
    return {
        "layernorm_fp8": (te.te_add_layernorm_fp8, dict(norm, fmt=te.E4M3, scale=one(), q_row=q(T, K), amax_out=one(),
                                                        scale_inv_out=one())),
        "layernorm_mxfp8": (te.te_add_layernorm_mxfp8, dict(norm, q_row=q(T, K), s_row=mx(T, K))),
        "layernorm_bwd": (te.te_layernorm_bwd, dict(dy=gpu(T, K), s=gpu(T, K), gamma=v(K), mu=v(T), rsigma=v(T), dx=gpu(T, K),
                                                    dgamma=v(K), dbeta=v(K), workspace=v(2 * T * K), dres=gpu(T, K), stream=7)),
        "bf16": (te.te_act_gemm_bf16, dict(res, x=gpu(T, K), w=gpu(N, K))),
        "fp8": (te.te_act_gemm_fp8, dict(out, x=q(T, K), fx=te.E4M3, w=q(N, K), fw=te.E4M3, x_scale_inv=one(), w_scale_inv=one(),
                                         q=q(T, N), q_scale=one(), q_amax=one(), q_scale_inv=one())),
        "mxfp8": (te.te_act_gemm_mxfp8, dict(out, x=q(T, K), sx=mx(T, K), w=q(N, K), sw=mx(N, K), q=q(T, N), s_q=mx(T, N))),
        "nvfp4": (te.te_act_gemm_nvfp4, dict(res, x=q(T, K // 2), sx=nv(T, K), gx=one(), w=q(N, K // 2), sw=nv(N, K), gw=one())),
        "dgrad_fp8": (te.te_act_dgrad_fp8, dict(grad, dy=q(T, K), fd=te.E5M2, w2=q(N, K), fw=te.E4M3, dy_scale_inv=one(),
                                                w2_scale_inv=one())),
        "dgrad_mxfp8": (te.te_act_dgrad_mxfp8, dict(grad, dy=q(T, K), sd=mx(T, K), w2=q(N, K), sw=mx(N, K))),
        "dgrad_nvfp4": (te.te_act_dgrad_nvfp4, dict(grad, dy=q(T, K // 2), sd=nv(T, K), gd=one(), w2=q(N, K // 2), sw=nv(N, K),
                                                    gw=one())),
        "bwd_bf16": (te.te_act_bwd_bf16, dict(grad, x=gpu(T, K), w=gpu(N, K), w2=gpu(48, N), dy=gpu(T, 48), dx=gpu(T, K),
                                              dw=gpu(N, K))),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_a_tensor_of_another_gpu_is_refused(library, name):  # noqa: F811
    fn, args = calls()[name]
    fn(**args)
    assert len(library.calls) == 1
    library.calls.clear()
    for key, value in args.items():
        if isinstance(value, torch.Tensor):
            for other in (gpu(*value.shape, dtype=value.dtype, index=1), torch.zeros(*value.shape, dtype=value.dtype)):
                with pytest.raises(ValueError, match=key):
                    fn(**{**args, key: other})
            with pytest.raises((TypeError, ValueError), match=key):
                fn(**{**args, key: gpu(*value.shape, dtype=torch.float16)})
    assert library.calls == []
