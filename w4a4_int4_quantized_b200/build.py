"""Build ``libw4a4.so`` (the C-ABI library) in-tree with nvcc for sm_100a.

Every translation unit under ``csrc/`` is compiled for ``sm_100a`` only (no
PTX for other targets, no other architectures), then linked into one shared
object next to this file, with the CUDA runtime linked statically so the
library loads on hosts without a GPU.  ``_calls.<torch>.<python>.so`` beside it
(``calls.cpp``, g++ against torch's headers) marshals the arguments of the
shortest calls; the C ABI needs neither it nor torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libw4a4.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "-I", INCLUDE,
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def calls_path() -> str:
    """The marshalling module for the running torch and Python: it has torch's C++
    tensor layout and CPython's API compiled in, so its name says which."""
    import sysconfig

    import torch
    return os.path.join(HERE, f"_calls.torch-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _build_calls(force: bool) -> None:
    try:
        import torch
    except ImportError:
        print("torch is not installed: the C ABI only, without the Python calls of calls.cpp", file=sys.stderr)
        return
    import sysconfig

    path = calls_path()
    deps = [CALLS_SRC, os.path.join(INCLUDE, "w4a4.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps):
        return
    root = os.path.dirname(torch.__file__)
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], CALLS_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), f"-Wl,-rpath,{os.path.join(root, 'lib')}",
           "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _build_library(verbose_ptxas: bool) -> None:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
           "--cudart", "static", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or _stale():
        _build_library(verbose_ptxas)
    _build_calls(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
