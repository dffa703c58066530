"""Builds the in-tree CUDA library libprism_b200.so for sm_100a with nvcc, and
_prism_bind.so, the cache calls' marshalling from PyTorch tensors, with g++.

Usage: python block_sparse_attention_band_b200/build.py [--force] [-v]
(run by path: importing the package requires the library this script builds)
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libprism_b200.so")
BIND = os.path.join(HERE, "_prism_bind.so")
SOURCES = ["prism.cu"]
DEPS = ["prism.cu", "estimate.cuh", "attention.cuh", "cache.cuh", "cache_attention.cuh", "cache_rows.cuh", "cache_tiles.cuh", "ptx.cuh"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libprism_b200.so")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def needs_build() -> bool:
    return _stale(LIB, [os.path.join(CSRC, d) for d in DEPS] + [os.path.join(ROOT, "include", "prism.h")])


def build_bind(force: bool = False) -> str | None:
    """Without PyTorch there are no tensors to marshal and nothing is built: the
    library, its C ABI and the calls that take addresses do without."""
    src = os.path.join(CSRC, "bind.cpp")
    if not force and not _stale(BIND, [src, os.path.join(ROOT, "include", "prism.h")]):
        return BIND
    import sysconfig

    try:
        import torch
    except ImportError:
        print("PyTorch is not installed: _prism_bind.so (the cache calls' marshalling) is not built", file=sys.stderr)
        return None
    base = os.path.dirname(torch.__file__)
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in (os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")):
        cmd += ["-isystem", d]
    cmd += [src, "-o", BIND + ".tmp", "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", f"-Wl,-rpath,{os.path.join(base, 'lib')}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(BIND + ".tmp", BIND)
    return BIND


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    cmd = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp"]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)  # (first: it does not need what the other part fails without)
    build_bind(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
