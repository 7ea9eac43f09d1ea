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
