"""The parts that a contraction is cut into, for the longest ones that the calls take: every k-tile is in one part, no part
is empty or longer than asked.  The ranges are compiled for the host; two calls whose products of k-tiles and segments
pass 2^31 run on the GPU."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import nvfp4_precision_transformer_gb300 as te
from tests import gpu_util as G
from tests.test_launch_setup import CSRC, CUDA

MAIN = r"""
#include <stdio.h>
#include "common.cuh"
#define CHECK(c) do { if (!(c)) { printf("line %d: %s (%d, %d)\n", __LINE__, #c, n, seg); return 1; } } while (0)
int main() {
  const int lengths[] = {1, 2, 12, 13, 14, 26, 27, 63, 64, 65, 129, 1000, 1 << 18, (1 << 19) - 1, 1 << 19, 8388593, 1 << 23, 1 << 24};
  for (int n : lengths)
    for (int seg : {13, 64}) {
      const int segs = (n + seg - 1) / seg;
      int at = 0;
      CHECK(te::part_begin(n, 0, segs) == 0);
      for (int s = 0; s < segs; ++s) {
        const int end = te::part_begin(n, s + 1, segs);
        CHECK(end > at && end - at <= seg);
        at = end;
      }
      CHECK(at == n);
    }
  return 0;
}"""


def test_every_k_tile_is_in_one_segment(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or CUDA is None:
        pytest.skip("no C++ compiler or no CUDA headers")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(MAIN)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-w", "-I", CSRC, "-I", os.path.join(CUDA, "include"), str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout + out.stderr


@pytest.mark.parametrize("name", ["gemm.cuh", "act_stream.cuh"])
def test_the_kernels_cut_by_it(name):
    """No product of k-tiles in 32 bits."""
    text = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
    assert text.count("part_begin(") >= 2
    assert not re.findall(r"\bk_(?:num|tiles) \* (?:sg|part|\()", text)


def test_a_product_in_32_bits_would_leave_k_tiles_out():
    """What the ranges were: 2^19 k-tiles in 2^13 segments."""
    n, segs = np.int32(2 ** 19), 2 ** 13
    s = np.arange(segs + 1, dtype=np.int32)
    with np.errstate(over="ignore"):
        at = (n * s).astype(np.int64)
    at = np.where(at < 0, -((-at) // segs), at // segs)       # as C divides
    assert np.clip(np.diff(at), 0, None).sum() < 2 ** 19 and (np.diff(at) <= 0).any()


@pytest.mark.gpu
def test_dgrad_of_a_long_contraction():
    """MXFP8, 2^26 columns of dy: 2^19 k-tiles in 2^13 segments.  Each row of W2 has a one in every k-tile."""
    N, F = 1 << 26, 16
    one = 0x38                                                   # E4M3 1.0; E8M0 127: 2^0
    d = torch.full((1, N), one, dtype=torch.uint8, device=G.DEV)
    w = torch.zeros(F, N // 128, 128, dtype=torch.uint8, device=G.DEV)
    for f in range(F):
        w[f, :, 8 * f + f % 8] = one
    s = torch.full((te.te_scale_bytes(te.E8M0, F, N),), 127, dtype=torch.uint8, device=G.DEV)
    dz = torch.zeros(1, F, dtype=torch.bfloat16, device=G.DEV)
    db = torch.zeros(F, device=G.DEV)
    ws = torch.empty(te.te_act_dbias_workspace_bytes(1, F) // 4, device=G.DEV)
    te.te_act_dgrad_mxfp8(d, s, w.view(F, N), s, None, te.ACT_NONE, dz, db, ws)
    torch.cuda.synchronize()
    G.check_no_device_error()
    assert bool((dz == N // 128).all()) and bool((db == N // 128).all())


@pytest.mark.gpu
def test_forward_of_a_long_contraction():
    """BF16, K = 2^27: the CTAs that share the tile have 2^18 k-tiles each, in 20165 segments."""
    K, N = 1 << 27, 16
    x = torch.ones(1, K, dtype=torch.bfloat16, device=G.DEV)
    w = torch.zeros(N, K // 64, 64, dtype=torch.bfloat16, device=G.DEV)
    for n in range(N):
        w[n, :, 4 * n + n % 4] = 1.0
    y = torch.zeros(1, N, device=G.DEV)
    te.te_act_gemm_bf16(x, w.view(N, K), te.ACT_NONE, y=y)
    torch.cuda.synchronize()
    G.check_no_device_error()
    assert bool((y == K // 64).all())
