"""Kernels that are set up beside the kernel before them read what it wrote with ordinary loads.

Such a kernel's life begins while the other one still writes, and a load by the read-only path
(``__ldg``, ``ld.global.nc``, a ``const __restrict__`` parameter) is defined only for data that
nobody writes while the kernel lives; the compiler may also move it above the wait.  So the files
whose kernels call ``pdl_wait`` have none, but for the bias, which only calls that are launched in
full stream order pass."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nvfp4_precision_transformer_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".inc")))


def _code(name):
    """The file's lines without comments."""
    text = open(os.path.join(CSRC, name)).read()
    return [re.sub(r"//.*", "", line) for line in text.splitlines()]


def _dependent(name):
    """Whether the file holds (part of) a kernel that waits for the one before it."""
    return name == "gated_epilogue.inc" or any("pdl_wait()" in line for line in _code(name))


def test_the_dependent_kernels_are_found():
    found = {f for f in FILES if _dependent(f)}
    assert {"norm.cu", "gemm.cuh", "gated_decode.cuh", "gated_stream.cuh", "gated_stream_block.cuh", "host.cu"} <= found


@pytest.mark.parametrize("name", [f for f in FILES if _dependent(f)])
def test_no_read_only_loads_behind_the_wait(name):
    bad = [(i + 1, line.strip()) for i, line in enumerate(_code(name))
           if re.search(r"__ldg\(|\.nc\b|__restrict__|__ldlu|__ldcs|__ldcg", line) and "args.bias" not in line]
    assert not bad, bad


def test_a_bias_comes_only_in_stream_order():
    """te_gemm_* pass the bias and no programmatic launch; the chained GEMM passes none."""
    gemm = " ".join(_code("gemm.cu"))
    chained = gemm[gemm.index("gemm_bf16_tokens("):gemm.index('extern "C"')]
    entries = gemm[gemm.index('extern "C"'):]
    assert "bias" not in chained and "pdl" in chained
    assert "bias" in entries and "Pdl" not in entries and "pdl" not in entries
    gated = " ".join(_code("gated.cu"))
    assert "bias" not in gated
