"""The first-call look-ups of the launchers (csrc/launch_setup.cuh), compiled for the host with stand-ins for
the CUDA runtime's functions."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_precision_transformer_gb300", "csrc")
CUDA = next((p for p in (os.environ.get("CUDA_HOME"), "/usr/local/cuda") if p and os.path.exists(p)), None)

STUBS = r"""
#include <stdio.h>
#include <string.h>
#include "launch_setup.cuh"

static int fail_cluster = 0, pending = 0, recorded = 0, attributes = 0, fail_attribute = 0;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { int p = pending; pending = 0; return static_cast<cudaError_t>(p); }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  if (fail_attribute) return static_cast<cudaError_t>(pending = cudaErrorInvalidValue);
  ++attributes;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* cfg) {
  const int size = static_cast<int>(cfg->attrs[0].val.clusterDim.x);
  if (size == fail_cluster) return static_cast<cudaError_t>(pending = cudaErrorInvalidClusterSize);
  *n = 152 / size;
  return cudaSuccess;
}
}
namespace te {
te_status record_cuda(cudaError_t e) { if (e != cudaSuccess) ++recorded; return e == cudaSuccess ? TE_OK : TE_ERR_CUDA; }
}
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
"""


def run(tmp_path, main, *flags):
    cxx = shutil.which("g++")
    if cxx is None or CUDA is None:
        pytest.skip("no C++ compiler or no CUDA headers")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(STUBS + main)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-w", *flags, "-I", CSRC, "-I", os.path.join(CUDA, "include"), str(src),
                        "-o", str(exe), "-pthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr


@pytest.mark.parametrize("size", [2, 4, 8])
def test_a_cluster_size_that_cannot_run_is_left_out(tmp_path, size):
    """The other forms still run: no error is returned, recorded or left behind."""
    run(tmp_path, r"""
int main() {
  fail_cluster = %d;
  te::StreamSetup s = {};
  CHECK(s.set(&s, &s, 192, 200000) == TE_OK);
  for (int i = 0; i < 3; ++i) CHECK(s.most[i] == ((2 << i) == fail_cluster ? 0 : 152 / (2 << i)));
  CHECK(pending == 0 && recorded == 0 && attributes == 2);
  return 0;
}""" % size)


def test_a_kernel_that_cannot_have_its_shared_memory_is_an_error(tmp_path):
    run(tmp_path, r"""
int main() {
  fail_attribute = 1;
  te::StreamSetup s = {};
  CHECK(s.set(&s, &s, 192, 200000) == TE_ERR_CUDA && recorded == 1 && pending == 0);
  fail_attribute = 0;   // and the next call tries again
  CHECK(s.set(&s, &s, 192, 200000) == TE_OK && s.most[2] == 19);
  return 0;
}""")
