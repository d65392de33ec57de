"""Build libfused_norm.so in-tree for sm_100a (B200).

    python -m rmsnorm_row_b200.build          # or: python rmsnorm_row_b200/build.py

Each .cu under csrc/ and csrc/block/ compiles on its own (in parallel) with
``-gencode arch=compute_100a,code=sm_100a``; the objects link into one shared
library with the CUDA runtime linked statically, so loading the library needs no
GPU and no CUDA shared libraries beyond the driver at launch time.
Precise division and square root are kept (no fast-math).

csrc/binding/ is the Python side of the operators of include/block_ops.h, a CPython extension
(_binding.so) against the installed PyTorch that links to the library. Without PyTorch only the
library is built, which is all that C programs need (the Python package needs PyTorch anyway).
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libfused_norm.so")
BINDING = os.path.join(HERE, "_binding.so")
BUILD_DIR = os.path.join(HERE, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    return obj


def _torch_is_installed() -> bool:
    return importlib.util.find_spec("torch") is not None


def _build_binding() -> None:
    import sysconfig

    import torch

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    root = os.path.dirname(torch.__file__)
    includes = [sysconfig.get_paths()["include"], os.path.join(root, "include"), os.path.join(cuda, "include")]
    libs = os.path.join(root, "lib")
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f for d in includes for f in ("-isystem", d)), os.path.join(CSRC, "binding", "block_ops.cpp"),
           "-o", tmp, LIB, "-L" + libs, "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"the binding does not compile:\n{res.stderr[-4000:]}")
    os.replace(tmp, BINDING)


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    srcs = glob.glob(os.path.join(CSRC, "**", "*"), recursive=True) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return any(os.path.getmtime(s) > t for s in srcs)


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int = 4) -> str:
    if force or _stale(LIB):
        os.makedirs(BUILD_DIR, exist_ok=True)
        srcs = sorted(glob.glob(os.path.join(CSRC, "**", "*.cu"), recursive=True))
        with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
        force = True
    if not _torch_is_installed():
        print("PyTorch is not installed: _binding.so is left out", file=sys.stderr)
    elif force or _stale(BINDING):
        _build_binding()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
