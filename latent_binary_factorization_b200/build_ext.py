"""Build liblittlebit.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_cache.so, the compiled marshalling of cache.py, beside it with g++."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "liblittlebit.so")
BINDING = os.path.join(HERE, "_cache.so")
SOURCES = ["littlebit_capi.cu", "pack.cu", "decode.cu", "prefill.cu", "init.cu", "noalloc.cu", "selfcheck.cu", "cache.cu",
           "attend.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def build(verbose: bool = False, force: bool = False) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, "lb_internal.h"), os.path.join(CSRC, "per_device.h"),
            os.path.join(INCLUDE, "littlebit.h")]
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(d) for d in deps)
        if os.path.getmtime(LIB) >= newest:
            return LIB
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-cudart", "static", "-I", INCLUDE, "-I", CSRC, *srcs, "-o", LIB]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stdout.write(res.stdout)
        sys.stderr.write(res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed with code {res.returncode}")
    return LIB


def build_binding(verbose: bool = False, force: bool = False) -> str:
    """_cache.so, linked against torch and liblittlebit.so (build() it first)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    src = os.path.join(CSRC, "cache_binding.cpp")
    deps = [src, os.path.join(INCLUDE, "littlebit.h")]
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(os.path.getmtime(d) for d in deps):
        return BINDING
    includes = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths(device_type="cuda")]
    libs = cpp_extension.library_paths(device_type="cuda")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in includes], src,
           "-o", BINDING, f"-L{HERE}", "-llittlebit", "-Wl,-rpath,$ORIGIN", *[f"-L{d}" for d in libs], "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd))
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stdout.write(res.stdout)
        sys.stderr.write(res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed with code {res.returncode}")
    return BINDING


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force=True)
    build_binding(verbose="-v" in sys.argv, force=True)
