"""Builds ``libkvq.so`` in-tree with nvcc for sm_103a (GB300).

Each .cu file compiles to an object in ``_build/`` (in parallel), then one
shared library is linked next to this file.  No fast-math: the encoders rely
on IEEE f32 division and square root and on the absence of fused
multiply-adds the source does not write.

Beside it, apart from it, the Python extension ``_paged_host.so`` (g++, the headers of
Python and PyTorch), which checks the tensors of the paged calls and is needed by them
alone.  It is built for one Python and one PyTorch: a stamp in ``_build/`` says which.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkvq.so")
HOST = os.path.join(HERE, "_paged_host.so")
HOST_STAMP = os.path.join(BUILD, "_paged_host.stamp")
HOST_SOURCE = os.path.join(CSRC, "paged_host.cpp")
HEADER = os.path.join(ROOT, "include", "kvq.h")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvq")


def flags() -> list[str]:
    return ["-O3", "-std=c++17", ARCH, "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-O3",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.inc")) + \
        [HEADER]


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _host_made_for() -> str:
    """What the extension's binary interface depends on."""
    import torch

    return "\n".join([f"torch {torch.__version__} {os.path.dirname(torch.__file__)}",
                      f"cxx11 abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                      f"python {sysconfig.get_config_var('EXT_SUFFIX')}"]) + "\n"


def host_up_to_date() -> bool:
    if not _newer(HOST, [HOST_SOURCE, HEADER]) or not os.path.exists(HOST_STAMP):
        return False
    with open(HOST_STAMP) as f:
        return f.read() == _host_made_for()


def up_to_date() -> bool:
    return library_up_to_date() and host_up_to_date()


def build_host(force: bool = False, verbose: bool = False) -> str:
    """The extension of the paged calls."""
    if not force and host_up_to_date():
        return HOST
    import torch

    os.makedirs(BUILD, exist_ok=True)
    made_for = _host_made_for()
    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    tmp = HOST + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in include), HOST_SOURCE,
           "-o", tmp, f"-L{os.path.join(base, 'lib')}", "-lc10", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{cmd[0]} failed on {HOST_SOURCE}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {HOST_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST)
    tmp = HOST_STAMP + f".{os.getpid()}.tmp"
    with open(tmp, "w") as f:
        f.write(made_for)
    os.replace(tmp, HOST_STAMP)
    return HOST


def build_library(force: bool = False, verbose: bool = False) -> str:
    """The kernels and their C entry points: nvcc alone."""
    if not force and library_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *flags(), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, ARCH, "-shared", "-o", tmp, *objs, "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """Both; the library is there even if the extension cannot be built (which raises)."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        host = ex.submit(build_host, force, verbose)
        path = build_library(force, verbose)
        host.result()
    return path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
