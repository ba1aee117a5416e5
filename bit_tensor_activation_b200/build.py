"""Compiles libhq.so (all CUDA kernels + the C ABI) in-tree for sm_100a, and the Python binding's
argument checks (_hqargs.so)."""
from __future__ import annotations

import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SO = os.path.join(PKG, "libhq.so")
ARGS_SO = os.path.join(PKG, "_hqargs.so")
SOURCES = [os.path.join(PKG, "csrc", "hq_api.cu")]
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-fmad=false",           # every float op stays one IEEE operation (bit-exact with the spec)
    "-Xcompiler", "-fPIC", "-shared",
]


def build(verbose: bool = False, extra_flags=()) -> str:
    cmd = ["nvcc", *NVCC_FLAGS, *extra_flags, "-I", os.path.join(ROOT, "include"), *SOURCES, "-o", SO]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    build_args(verbose)
    return SO


def build_args(verbose: bool = False) -> str:
    """_hqargs.so: a Python module over libhq.so and torch's own headers and libraries."""
    import torch
    from torch.utils import cpp_extension

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    include = [f"-I{p}" for p in (os.path.join(ROOT, "include"), *cpp_extension.include_paths("cuda"),
                                  sysconfig.get_paths()["include"])]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *include,
           os.path.join(PKG, "csrc", "hq_args.cpp"), "-o", ARGS_SO, f"-L{PKG}", "-l:libhq.so",
           f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    return ARGS_SO


if __name__ == "__main__":
    build(verbose=True)
