"""Build libvsa_gb300.so (the CUDA kernels + C ABI) in-tree with nvcc for sm_103a.

    python -m block_sparse_attention_vsa_gb300.build [--force]

Two translation units compiled side by side, one -gencode (sm_103a), static CUDA runtime,
no cmake.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libvsa_gb300.so")
SOURCES = [os.path.join(CSRC, f) for f in ("vsa_api.cu", "vsa_serve_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in (
    "vsa_fwd_kernel.cuh", "vsa_bwd_kernel.cuh", "vsa_select_kernel.cuh", "vsa_cache_kernel.cuh",
    "sm103_ptx.cuh", "vsa_warp_ptx.cuh", "vsa_host.h")] + [
    os.path.join(ROOT, "include", "vsa.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-shared", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr", "--threads", "2"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libvsa_gb300.so")


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS if os.path.exists(p))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + SOURCES + [
        "-o", tmp, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
