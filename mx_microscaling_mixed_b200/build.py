"""Builds libmxs.so (all CUDA sources under csrc/) in-tree for sm_100a, and the
native half of the Python binding (csrc/binding.cpp), an extension for one
torch and Python.  The library is what the calls need; without the extension
the binding goes its general way.

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
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                 "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def binding_path() -> str:
    """The extension for the torch and Python at hand: compiled against both,
    so that it is never loaded by others."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_binding-torch{torch.__version__}-abi{int(torch.compiled_with_cxx11_abi())}"
                        + sysconfig.get_config_var("EXT_SUFFIX"))


def _stale(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


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


def _link_binding(obj: str, path: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = path + f".tmp{os.getpid()}"
    subprocess.check_call([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libmxs.so",
                           "-Wl,-rpath,$ORIGIN", "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    header = os.path.join(ROOT, "include", "mxs.h")
    path = binding_path()
    lib = force or _stale(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [header])
    ext = force or _stale(path, [os.path.join(CSRC, "binding.cpp"), header])
    if not lib and not ext:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    obj = os.path.join(OBJ, "binding.o")
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        done = ex.submit(_compile_binding, obj) if ext else None
        if lib:
            objs = list(ex.map(_compile, _sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
            os.replace(tmp, LIB)
    if ext:
        try:
            done.result()
            _link_binding(obj, path)
        except (subprocess.CalledProcessError, OSError) as e:
            # (an extension of older sources would see another ABI than the library's)
            if os.path.exists(path):
                os.remove(path)
            print(f"{os.path.basename(path)} not built ({e}): calls go through ctypes alone", file=sys.stderr)
    if verbose:
        print("built", LIB, *([path] if os.path.exists(path) else []))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
