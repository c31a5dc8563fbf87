"""Builds libquarot.so in-tree for sm_103a with nvcc (no CMake, no torch), and
beside it the Python module of the 8-bit and the paged calls (host code against torch), which
the package can do without: where it cannot be built, a warning says so.

Each translation unit under csrc/ is compiled in parallel, as relocatable
device code or (WHOLE_PROGRAM) by itself, then linked into a shared library next to this file.  A rebuild is
skipped when what it gives is newer than every source and header.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libquarot.so")
CALLS_SRC = os.path.join(CSRC, "fp8_calls.cpp")
CALLS_HEADER = os.path.join(CSRC, "paged_calls.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
WHOLE_PROGRAM = {"fp8_gemm.cu"}  # ptxas honours setmaxnreg only there
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libquarot.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def calls_path() -> str:
    """Where the Python module of the 8-bit calls belongs: it fits one Python, one torch and one C++ ABI of it, which its
    name states, so that another one's is never loaded."""
    import torch

    tag = f"{sys.implementation.cache_tag}-torch{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(HERE, f"_fp8_calls.{tag}.so")


def _newer(target: str, sources) -> bool:
    common = [os.path.join(ROOT, "include", "quarot.h"), os.path.abspath(__file__)]
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in [*sources, *common])


def _lib_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")))


def _calls_up_to_date() -> bool:
    try:
        return _newer(calls_path(), [CALLS_SRC, CALLS_HEADER])
    except ImportError:  # no torch: nothing to build it against
        return False


def up_to_date() -> bool:
    return _lib_up_to_date() and _calls_up_to_date()


def _build_calls(nvcc: str) -> None:
    """The Python module of the 8-bit calls; torch is loaded before it, so its libraries need no path."""
    import torch

    t = os.path.dirname(torch.__file__)
    path = calls_path()
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DUSE_CUDA",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(t, "include"),
           "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"), CALLS_SRC, "-o", tmp,
           "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(CALLS_SRC)}:\n{r.stderr}")
    os.replace(tmp, path)


def _try_calls(nvcc: str) -> None:
    try:
        _build_calls(nvcc)
    except Exception as e:  # no torch, no g++, no headers of either: the library needs none of them
        warnings.warn(f"the compiled 8-bit calls were not built, the general path takes them: {e}", RuntimeWarning)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path.  Raises on any nvcc error."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    if not force and _lib_up_to_date():
        _try_calls(nvcc)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        rdc = "-rdc=false" if os.path.basename(src) in WHOLE_PROGRAM else "-rdc=true"
        cmd = [nvcc, *ARCH, *FLAGS, rdc, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return r.stderr

    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        calls = ex.submit(_try_calls, nvcc) if force or not _calls_up_to_date() else None
        logs = list(ex.map(compile_one, zip(srcs, objs)))
        if calls is not None:
            calls.result()
    if verbose:
        for log in logs:
            if log.strip():
                print(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-rdc=true", "--cudart=static", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
