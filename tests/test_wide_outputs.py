"""fp32 outputs so wide that a row's bytes pass 2^31 are refused: the kernels count columns in bytes, in 32 bits.  Runs on
the CPU; nothing is enqueued."""
import ctypes

import nvfp4_precision_transformer_gb300 as te

OK = ctypes.c_void_p(0x1000)     # never dereferenced
SHAPE = 2
WIDE, MOST = (1 << 29) + 16, 1 << 29


def test_weight_gradient_of_the_activation():
    def bwd(K, dt, accumulate):
        return te.lib().te_act_bwd_bf16(OK, OK, OK, OK, OK, te.ACT_GELU, OK, None, None, 0, OK, OK, dt, accumulate, 4, K, 32, 32, None)

    for accumulate in (0, 1):
        assert bwd(WIDE, te.F32, accumulate) == SHAPE
    assert bwd((1 << 30) + 16, te.BF16, 0) == SHAPE


def test_gemms():
    L, F32 = te.lib(), te.F32
    assert L.te_gemm_bf16(OK, 0, OK, 0, None, OK, F32, 0, 16, WIDE, 32, None) == SHAPE
    assert L.te_gemm_fp8(OK, te.E4M3, OK, te.E4M3, OK, OK, None, OK, F32, 0, 16, WIDE, 32, None) == SHAPE
    assert L.te_gemm_mxfp8(OK, te.E4M3, OK, OK, te.E4M3, OK, None, OK, F32, 0, 16, WIDE, 32, None) == SHAPE
    assert L.te_gemm_nvfp4(OK, OK, OK, OK, OK, OK, None, OK, F32, 0, 16, WIDE, 32, None) == SHAPE
    for n, dt, acc in ((MOST, F32, 0), (WIDE, F32, 1), (WIDE, te.BF16, 0)):      # past the sizes, up to the missing operand
        assert L.te_gemm_bf16(None, 0, OK, 0, None, OK, dt, acc, 16, n, 32, None) == 1


def test_weight_gradient_of_the_gated_projections():
    bwd = te.lib().te_gated_bwd_bf16
    assert bwd(OK, OK, OK, OK, OK, te.ACT_SILU, OK, OK, OK, te.F32, 0, 4, WIDE, 32, 32, None) == SHAPE
