"""Build ``libfp8bw.so`` (the C-ABI library) in-tree with nvcc for sm_100a, and then, where
torch is installed, ``_calls.so`` (the Python binding's compiled calls) with g++.

Usage: ``python -m blockwise_fp8_linear_b200.build [--force] [--verbose]``.
Rebuilds only when a source or header is newer than the library.  IEEE division and
no flush-to-zero are required for bit-exact quantization, so no fast-math flags.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfp8bw.so")
CALLS = os.path.join(HERE, "_calls.so")
BUILD_DIR = os.path.join(HERE, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-prec-div=true",
              "-ftz=false", "-prec-sqrt=true", "-fmad=true", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfp8bw")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def build_calls(force: bool = False) -> str:
    """The compiled calls; rebuilt when their source, the header or torch is newer."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    src = os.path.join(CSRC, "calls.cpp")
    deps = [src, os.path.join(INCLUDE, "fp8bw.h"), torch.__file__, __file__]
    if not force and os.path.exists(CALLS) and \
            all(os.path.getmtime(p) <= os.path.getmtime(CALLS) for p in deps):
        return CALLS
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths(),
           os.path.join(cuda, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + f".tmp{os.getpid()}"
    subprocess.run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                    "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                    *[f"-I{i}" for i in inc], src, "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch",
                    "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, CALLS)
    return CALLS


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB):
        t = os.path.getmtime(LIB)
        if all(os.path.getmtime(p) <= t for p in _deps()):
            return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"], check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """The library first: C programs need neither torch nor its headers."""
    build_library(force, verbose)
    if importlib.util.find_spec("torch") is not None:
        build_calls(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
