"""Build libte_gb300.so in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel; the quantizer unit is compiled
with -fmad=false so that no multiply-add is contracted in code-deciding
arithmetic.  The result lands next to this file and is git-ignored.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libte_gb300.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--cudart", "shared"]
UNITS = {"host.cu": [], "quant.cu": ["-fmad=false"], "norm.cu": [], "layernorm.cu": [], "gemm.cu": [], "gated.cu": [],
         "act.cu": ["-Xptxas", "-v"]}


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def check_registers(log: str) -> int:
    """The kernels whose warps hand registers to one another (gemm_kernel with the epilogues kAct and kActGrad) have the
    number at launch that their split adds up to: with another one the launcher would refuse every call.  ``log`` is what
    ptxas -v says; returns how many such kernels there are."""
    with open(os.path.join(CSRC, "gemm.cuh")) as f:
        want = int(re.search(r"kLaunchRegs = (\d+)", f.read())[1])
    found = re.findall(r"Compiling entry function '(\S*gemm_kernelILi\dELi2ELi[34]E\S*)'.*?Used (\d+) registers", log, re.S)
    bad = [f"{name}: {n}" for name, n in found if int(n) != want]
    if bad or not found:
        raise RuntimeError(f"registers at launch other than {want}: {bad or 'no such kernel found'}")
    return len(found)


def build(verbose: bool = False, out_dir: str | None = None) -> str:
    nvcc = _nvcc()
    obj_dir = out_dir or os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)

    def compile_one(unit):
        src = os.path.join(CSRC, unit)
        obj = os.path.join(obj_dir, unit.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *COMMON, *UNITS[unit], "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {unit}:\n{r.stderr}")
        if unit == "act.cu":
            check_registers(r.stderr)
        if verbose:
            print(" ".join(cmd))
        return obj

    with ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
        objs = list(ex.map(compile_one, UNITS))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "--cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
