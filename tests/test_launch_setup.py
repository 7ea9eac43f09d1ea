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

static int fail_cluster = 0, pending = 0, recorded = 0, attributes = 0, no_room = 0, fail_attribute = 0;
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
  if (no_room) return *n = 0, cudaSuccess;
  *n = 152 / size;
  return cudaSuccess;
}
}
namespace te {
int num_sms() { return 152; }
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


THREADS = r"""
#include <thread>
#include <vector>
struct State { int a, b; };
int main() {
  for (int round = 0; round < 200; ++round) {
    te::PerDevice<State>* p = new te::PerDevice<State>;
    std::atomic<int> made{0}, wrong{0};
    std::vector<std::thread> t;
    for (int i = 0; i < 8; ++i)
      t.emplace_back([&] {
        te_status s = TE_OK;
        const State* v = p->get(&s, [&](State* m) { made++; m->a = round; m->b = ~round; return TE_OK; });
        if (v == nullptr || s != TE_OK || v->a != round || v->b != ~round) wrong++;
      });
    for (auto& x : t) x.join();
    CHECK(made == 1 && wrong == 0);
    delete p;
  }
  return 0;
}"""


def test_first_call_state_is_published_whole(tmp_path):
    """Eight threads make the first call at once: one looks up, all see its state complete; under the thread
    sanitizer where the compiler has one."""
    run(tmp_path, THREADS)
    probe = tmp_path / "p.cpp"
    probe.write_text("int main() { return 0; }")
    r = subprocess.run([shutil.which("g++"), "-fsanitize=thread", str(probe), "-o", str(tmp_path / "p")], capture_output=True)
    if r.returncode == 0 and subprocess.run([str(tmp_path / "p")], capture_output=True).returncode == 0:
        run(tmp_path, THREADS, "-fsanitize=thread")


def test_a_failed_look_up_is_tried_again(tmp_path):
    run(tmp_path, r"""
int main() {
  static te::PerDevice<int> p;
  te_status s = TE_OK;
  CHECK(p.get(&s, [](int* v) { *v = 3; return TE_ERR_CUDA; }) == nullptr && s == TE_ERR_CUDA);
  const int* v = p.get(&s, [](int* v) { *v = 4; return TE_OK; });
  CHECK(v != nullptr && *v == 4 && p.get(&s, [](int*) { return TE_ERR_CUDA; }) == v);
  return 0;
}""")


def test_no_launcher_has_a_plain_flag():
    """First-call state is reached through PerDevice (or under the lock of host.cu), never by an unguarded static."""
    for name in sorted(os.listdir(CSRC)):
        lines = [line.split("//")[0] for line in open(os.path.join(CSRC, name))]
        bad = [line.strip() for line in lines if line.lstrip().startswith("static ") and ("[64]" in line or " bool " in line)
               and "PerDevice" not in line and "constexpr" not in line and "(" not in line]
        assert not bad, (name, bad)


def test_gemm_pairs_that_cannot_run_are_an_error(tmp_path):
    """No CTA pair fits, and the query itself says nothing: the call must not return as if it had been made."""
    run(tmp_path, r"""
int main() {
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t cfg = {};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  te::GemmSetup g = {};
  attr[0].val.clusterDim = {2, 1, 1};
  CHECK(g.set(&g, 2, false, 200000, cfg) == TE_OK && g.units == 76);
  no_room = 1;
  CHECK(g.set(&g, 2, false, 200000, cfg) == TE_ERR_CUDA && recorded == 1);
  no_room = 0, fail_cluster = 2;
  CHECK(g.set(&g, 2, false, 200000, cfg) == TE_ERR_CUDA && recorded == 2 && pending == 0);
  // shared tiles: sizes that cannot run are only not taken
  fail_cluster = 8;
  CHECK(g.set(&g, 2, true, 200000, cfg) == TE_OK && g.units == 38 && g.fours == 0 && pending == 0);
  fail_cluster = 0, no_room = 1;
  CHECK(g.set(&g, 2, true, 200000, cfg) == TE_OK && g.units == 0 && g.fours == 0);
  return 0;
}""")
