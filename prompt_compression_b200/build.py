"""Build libspeckv.so (the sm_100a kernels behind include/speckv.h) and the
compiled part of the Python binding (_bind, csrc/bind.cpp) in-tree.

    python -m prompt_compression_b200.build [--force]

nvcc cross-compiles for sm_100a; no GPU is needed to build.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libspeckv.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(ROOT, "include", "speckv.h"), os.path.abspath(__file__)]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into prompt_compression_b200/libspeckv.so, and the binding."""
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(p) for p in _inputs())
        if os.path.getmtime(LIB) >= newest:
            build_binding(verbose=verbose)
            return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + NVCC_FLAGS + ["-o", tmp] + sources()
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd, cwd=PKG)
    os.replace(tmp, LIB)
    build_binding(force=force, verbose=verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/bind.cpp against torch's headers into prompt_compression_b200/_bind.so."""
    inputs = [BIND_SRC, os.path.join(ROOT, "include", "speckv.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(BIND) and os.path.getmtime(BIND) >= max(os.path.getmtime(p) for p in inputs):
        return BIND
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-o", tmp, BIND_SRC, "-L", PKG, "-l:libspeckv.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd, cwd=PKG)
    os.replace(tmp, BIND)
    return BIND


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
