"""Build libvsa_gb300.so (the CUDA kernels + C ABI) in-tree with nvcc for sm_103a, and
_vsa_torch_<torch>_<python>.so (the short way from torch tensors to its microsecond calls)
with g++.

    python -m block_sparse_attention_vsa_gb300.build [--force]

Three translation units compiled side by side, one -gencode (sm_103a), static CUDA runtime,
no cmake.
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libvsa_gb300.so")
SOURCES = [os.path.join(CSRC, f) for f in ("vsa_api.cu", "vsa_serve_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in (
    "vsa_fwd_kernel.cuh", "vsa_bwd_kernel.cuh", "vsa_select_kernel.cuh", "vsa_cache_kernel.cuh",
    "sm103_ptx.cuh", "vsa_warp_ptx.cuh", "vsa_host.h")] + [
    os.path.join(ROOT, "include", "vsa.h")]
TORCH_SOURCE = os.path.join(CSRC, "vsa_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-shared", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr", "--threads", "2"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libvsa_gb300.so")


def stale(lib: str = LIB, deps=None) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in (deps or DEPS) if os.path.exists(p))


def _torch_dir():
    """The directory of the torch that this Python imports (looked up without importing it),
    or None: the library itself builds without one."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec else None


def torch_lib(version: str) -> str:
    """The extension's file for this version of torch and this Python.  It is compiled against
    the layout of torch's own objects, so each pair has a file of its own."""
    tag = re.sub(r"[^0-9A-Za-z]+", "_", f"{version} {sysconfig.get_config_var('SOABI')}")
    return os.path.join(PKG, f"_vsa_torch_{tag}.so")


def _torch_command(torch_dir: str, out: str):
    """The g++ command for the extension, against that torch's headers and libraries."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(torch_dir, "include"), sysconfig.get_paths()["include"],
               os.path.join(cuda, "include")]
    return (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", TORCH_SOURCE]
            + [x for d in include for x in ("-isystem", d)]
            + ["-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
               "-ltorch_cuda", "-ltorch_python", "-ldl", "-o", out])


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is older than its sources.  Compilers are looked for only then."""
    jobs = []
    if force or stale():
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + SOURCES + [
            "-o", tmp, "-cudart", "static"]
        jobs.append((cmd, tmp, LIB))
    torch_dir = _torch_dir()
    if torch_dir:
        version = os.path.join(torch_dir, "version.py")
        with open(version) as f:
            said = re.search(r"^__version__ *= *['\"](.+?)['\"]", f.read(), re.M)
        lib = torch_lib(said.group(1))
        if force or stale(lib, [TORCH_SOURCE, DEPS[-1], version]):
            tmp = lib + ".tmp%d" % os.getpid()
            jobs.append((_torch_command(torch_dir, tmp), tmp, lib))
    running = [subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
               for cmd, _, _ in jobs]
    said = [p.communicate()[0] for p in running]
    for p, text, (cmd, tmp, lib) in zip(running, said, jobs):
        if p.returncode != 0:
            raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + text)
        if verbose:
            sys.stderr.write(text)
        os.replace(tmp, lib)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
