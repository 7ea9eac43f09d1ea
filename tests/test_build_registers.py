"""The build refuses kernels whose registers at launch are not those that their warps share out.  Runs on the CPU."""
import pytest

from nvfp4_precision_transformer_gb300 import build

LOG = """ptxas info    : 0 bytes gmem
ptxas info    : Compiling entry function '_ZN2te12_GLOBAL__N__11gemm_kernelILi0ELi2ELi4ELb0EEEv14CUtensorMap_st' for 'sm_103a'
ptxas info    : Function properties for _ZN2te12_GLOBAL__N__11gemm_kernelILi0ELi2ELi4ELb0EEEv14CUtensorMap_st
    96 bytes stack frame, 104 bytes spill stores, 184 bytes spill loads
ptxas info    : Used {a} registers, used 1 barriers, 96 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN2te12_GLOBAL__N__16act_dbias_kernelEPKfllPfi' for 'sm_103a'
ptxas info    : Used 57 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN2te12_GLOBAL__N__11gemm_kernelILi3ELi2ELi3ELb0EEEv14CUtensorMap_st' for 'sm_103a'
ptxas info    : Used {b} registers, used 1 barriers
"""


def test_the_split_adds_up():
    assert build.check_registers(LOG.format(a=168, b=168)) == 2


@pytest.mark.parametrize("a,b", [(160, 168), (168, 128), (255, 255)])
def test_another_count_is_an_error(a, b):
    with pytest.raises(RuntimeError, match="168"):
        build.check_registers(LOG.format(a=a, b=b))


def test_a_log_without_the_kernels_is_an_error():
    with pytest.raises(RuntimeError, match="no such kernel"):
        build.check_registers("ptxas info    : 0 bytes gmem\n")


def test_the_unit_is_compiled_with_the_log():
    assert "-v" in build.UNITS["act.cu"]
