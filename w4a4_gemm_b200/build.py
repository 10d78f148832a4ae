"""Build the sm_100a shared library ``libsvdq.so`` in-tree with nvcc, and the
CPython module ``svdq_torch`` (the cache operators' calls) beside it with g++.

    python -m w4a4_gemm_b200.build          # or: python w4a4_gemm_b200/build.py

The library is one translation unit (``csrc/svdq_api.cu``) compiled for
``sm_100a`` only, with the CUDA runtime linked statically and cuBLAS /
cuSOLVER (used once, during weight preparation) linked dynamically.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libsvdq.so")
TORCH_SRC = os.path.join(CSRC, "svdq_torch.cpp")
TORCH_LIB = os.path.join(HERE, "svdq_torch" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
            if f.endswith((".cu", ".cuh"))] + [os.path.join(INCLUDE, "svdq.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in _sources())


def torch_up_to_date() -> bool:
    if not os.path.exists(TORCH_LIB):
        return False
    t = os.path.getmtime(TORCH_LIB)
    return all(os.path.getmtime(s) <= t for s in (TORCH_SRC, os.path.join(INCLUDE, "svdq.h")))


def build_torch(force: bool = False, verbose: bool = False) -> str:
    """The CPython module: host code only, against torch's headers, linked to libsvdq.so beside it."""
    if not force and torch_up_to_date():
        return TORCH_LIB
    import torch
    from torch.utils import cpp_extension as E
    cuda_home = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    includes = E.include_paths() + [os.path.join(cuda_home, "include"), sysconfig.get_paths()["include"]]
    lib_dir = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in includes], TORCH_SRC, "-o", tmp, f"-L{HERE}", "-l:libsvdq.so", f"-L{lib_dir}",
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, TORCH_LIB)
    return TORCH_LIB


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        build_torch(verbose=verbose)
        return LIB
    nvcc = _nvcc()
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC,-fvisibility=hidden", "-cudart", "static",
           "-I", INCLUDE, os.path.join(CSRC, "svdq_api.cu"), "-o", tmp,
           "-L", cuda_lib, "-lcusolver", "-lcublas",
           f"-Xlinker=-rpath,{cuda_lib}"]
    if ptxas_info:
        cmd.insert(1, "-Xptxas=-v")
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    build_torch(verbose=verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
