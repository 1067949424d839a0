"""Builds libfl_int4g.so in-tree with nvcc for sm_103a (one -gencode).

Translation units are compiled in parallel, then linked into one shared
library (static CUDA runtime).  Rebuilds only when a source is newer than the
library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfl_int4g.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Kernels that split the registers of their launch among their warps, and the
# count a thread that the split adds up to.  They refuse to be launched with
# another one, so a compiler that chooses one is found here, when it builds.
REGISTERS = {"fl_kv8_prompt.cu": ("k_kv8_prompt", 96), "fl_int8_gemm.cu": ("k_int8_gemm", 96)}
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc():
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the int4g CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def check_registers(log, kernel, count):
    """Raises unless every build of `kernel` in a ptxas -v log has `count` registers."""
    used = {}
    for name, regs in re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", log, flags=re.S):
        if kernel in name:
            used[name] = int(regs)
    wrong = {n: r for n, r in used.items() if r != count}
    if wrong or not used:
        raise RuntimeError(f"{kernel} has to be compiled to {count} registers a thread, got {wrong or 'no such kernel'}: "
                           "its split of them among the warps has to be changed with the compiler")


def build(force=False, verbose=False):
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        split = REGISTERS.get(os.path.basename(src))
        cmd = [nvcc, *ARCH, *FLAGS, *(["-Xptxas", "-v"] if split else []), "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if split:
            check_registers(r.stdout + r.stderr, *split)
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
