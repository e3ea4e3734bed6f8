"""Build libdg.so (the CUDA kernels behind include/dg.h) in-tree for sm_103a.

Each translation unit is compiled by its own nvcc process, in parallel, then linked into
``entropy_bounded_denoising_gb300/_build/libdg.so``; beside it ``dg_bind-*.so``, the serving calls'
Python module (host code against Python's and PyTorch's headers; where they are missing the library is
built all the same, with a warning, and only the serving calls' Python forms are closed).  Either is
rebuilt only when one of its sources or headers is newer.
"""
from __future__ import annotations

import concurrent.futures
import contextlib
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libdg.so")
BIND = os.path.join(OUT, f"dg_bind-{torch.__version__}-{sys.implementation.cache_tag}.so")   # of one PyTorch and Python
BIND_SRC = os.path.join(CSRC, "dg_bind.cpp")
TORCH = os.path.dirname(os.path.abspath(torch.__file__))
HEADER = os.path.join(ROOT, "include", "dg.h")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _cuda() -> str:
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _nvcc() -> str:
    cand = os.path.join(_cuda(), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(target: str, deps: list[str]) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target)
                                             for p in deps + [HEADER, __file__])


def build_bind() -> str:
    """The serving calls' Python module; raises with the compiler's message where it cannot be built."""
    os.makedirs(OUT, exist_ok=True)
    tmp = BIND + f".tmp{os.getpid()}"
    lib = os.path.join(TORCH, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(TORCH, "include"), "-isystem", os.path.join(_cuda(), "include"),
           "-isystem", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"), BIND_SRC, "-o", tmp,
           "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"g++ failed for {BIND_SRC}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    return BIND


def _try_bind() -> None:
    try:
        build_bind()
    except RuntimeError as e:
        with contextlib.suppress(FileNotFoundError):
            os.remove(BIND)   # an older one, whose calls may not be the library's
        warnings.warn(f"the serving calls' Python module was not built: {e}", stacklevel=3)


def build(force: bool = False, verbose: bool = False) -> str:
    bind_stale = force or _stale(BIND, [BIND_SRC])
    if not force and not _stale(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh"))):
        if bind_stale:
            _try_bind()
        return LIB
    os.makedirs(OUT, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources()) + 1) as ex:
        bind = ex.submit(_try_bind) if bind_stale else None
        objs = list(ex.map(compile_one, sources()))
        if bind:
            bind.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs,
           "-Xcompiler", "-fPIC", "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
