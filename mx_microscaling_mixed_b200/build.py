"""Builds libmxs.so (all CUDA sources under csrc/) in-tree for sm_100a, and
_binding.so, the native half of the Python binding (csrc/binding.cpp).

    python -m mx_microscaling_mixed_b200.build [--force]

nvcc cross-compiles without a GPU.  The library is linked against the static
CUDA runtime and resolves driver entry points (tensor-map encoding) at run
time, so loading it needs no libcuda at link time.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmxs.so")
BINDING = os.path.join(PKG, "_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                 "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [os.path.join(CSRC, "binding.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "mxs.h")]


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    subprocess.check_call([NVCC, *CFLAGS, "-c", src, "-o", obj])
    return obj


def _compile_binding(obj: str) -> None:
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    abi = int(torch.compiled_with_cxx11_abi())
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
                           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
                           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
                           "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    subprocess.check_call([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libmxs.so",
                           "-Wl,-rpath,$ORIGIN", "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    binding = os.path.join(OBJ, "binding.o")
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        done = ex.submit(_compile_binding, binding)
        objs = list(ex.map(_compile, _sources()))
        done.result()
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    _link_binding(binding)
    if verbose:
        print("built", LIB, BINDING)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
