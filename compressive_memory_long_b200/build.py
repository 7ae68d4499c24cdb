"""Build in-tree: the CUDA library with nvcc for sm_100a (B200) only, and the Python entry of the
paged operators (a CPython extension over torch's headers) with g++."""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libinfini_attn.so")
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


def ext_path() -> str:
    """The extension's file, named after the interpreter and the torch it is built against: another
    torch finds none and builds its own, instead of loading one of another ABI."""
    import torch
    return os.path.join(PKG, f"_paged.{sys.implementation.cache_tag}-torch-{torch.__version__}.so")


def build_ext(force: bool = False, verbose: bool = False) -> str:
    """The CPython extension ``_paged``; it links the CUDA library next to it."""
    deps = [EXT_SRC, os.path.join(INCLUDE, "infini_attn.h"), os.path.abspath(__file__)]
    ext = ext_path()
    if not force and os.path.exists(ext) and all(os.path.getmtime(f) <= os.path.getmtime(ext) for f in deps):
        return ext
    import torch
    from torch.utils import cpp_extension as ce
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"), *ce.include_paths()]
    tmp = ext + f".tmp{os.getpid()}"
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
    os.replace(tmp, ext)
    return ext


def load_ext():
    """The extension module, built first where it is missing (not with INFINI_NO_AUTOBUILD=1)."""
    path = ext_path()
    if not os.path.exists(path):
        if os.environ.get("INFINI_NO_AUTOBUILD") == "1":
            raise ImportError(f"{path} is not built (python -m {__package__}.build)")
        build_ext()
    spec = importlib.util.spec_from_file_location(f"{__package__}._paged", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_ext(force=True, verbose=True))
