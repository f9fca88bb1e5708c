"""Build the in-tree CUDA library ``liblla.so`` for sm_100a with nvcc, and the Python
binding ``_binding.so`` of its later calls with g++.

Objects go to ``_build/`` at the repository root; the shared libraries are written
next to this file so that they travel with the package.  Rebuilds are
incremental on source/header modification times.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblla.so")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding.txt")    # what _binding.so was built for, and how
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build liblla.so")
    return path


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                     glob.glob(os.path.join(ROOT, "include", "*.h")))
    hdr_time = _newest(headers) if headers else 0.0
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_time)):
            continue
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    build_binding(verbose, force)
    return LIB


def build_binding(verbose: bool = False, force: bool = False) -> str:
    import torch
    from torch.utils.cpp_extension import include_paths

    src = os.path.join(CSRC, "binding.cpp")
    header = os.path.join(ROOT, "include", "lla.h")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [os.path.join(ROOT, "include"), *include_paths(), os.path.join(cuda, "include"),
            sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in dirs), src, "-o", BINDING,
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-L" + PKG,
           "-Wl,-rpath,$ORIGIN", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda",
           "-lc10", "-lc10_cuda", "-l:liblla.so"]
    # it holds for one torch and one Python only
    made_for = "\n".join([torch.__version__, sys.version, *cmd])
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING_FOR):
        with open(BINDING_FOR) as f:
            same = f.read() == made_for
        if same and os.path.getmtime(BINDING) >= _newest([src, header]):
            return BINDING
    if verbose:
        print(" ".join(cmd))
    if os.path.exists(BINDING_FOR):
        os.remove(BINDING_FOR)
    subprocess.run(cmd, check=True)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_FOR, "w") as f:
        f.write(made_for)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True))
