"""Build in-tree: the CUDA library with nvcc for sm_100a (B200) only, and the Python entry of the
paged operators (a CPython extension over torch's headers) with g++."""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libinfini_attn.so")
EXT = os.path.join(PKG, "_paged.so")
EXT_SRC = os.path.join(CSRC, "py_paged.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "--threads", "0",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(f) > t for f in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def build_ext(force: bool = False, verbose: bool = False) -> str:
    """The CPython extension ``_paged``; it links the CUDA library next to it."""
    deps = [EXT_SRC, os.path.join(INCLUDE, "infini_attn.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(EXT) and all(os.path.getmtime(f) <= os.path.getmtime(EXT) for f in deps):
        return EXT
    import torch
    from torch.utils import cpp_extension as ce
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"), *ce.include_paths()]
    tmp = EXT + f".tmp{os.getpid()}"
    # the system's g++, whose libstdc++ is the shared one torch uses: a compiler that links its own
    # copy would throw exceptions that the other copy's handlers cannot take
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for d in dirs for x in ("-isystem" if d != INCLUDE else "-I", d)], EXT_SRC, "-o", tmp,
           "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, EXT)
    return EXT


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_ext(force=True, verbose=True))
