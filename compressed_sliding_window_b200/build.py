"""Build libhca.so in-tree with nvcc for sm_100a, and with g++ the module that makes
the binding's paged calls (csrc/paged_calls.cpp, linked against it and torch).

Usage:  python -m compressed_sliding_window_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libhca.so")
MAIN_SRC = os.path.join(CSRC, "hca_lib.cu")
CALLS_PATH = os.path.join(PKG_DIR, "_paged_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
CALLS_SRC = os.path.join(CSRC, "paged_calls.cpp")
CALLS_STAMP = CALLS_PATH + ".stamp"     # what CALLS_PATH was built against

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libhca.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "hca.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    lib_m = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(s) <= lib_m for s in _sources())


def _built_against() -> str:
    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sys.version.split()[0]}\n")


def calls_up_to_date() -> bool:
    """Newer than its sources, and built against the torch and Python that run: the module uses
    torch's C++ interface, which another version need not share."""
    if not os.path.exists(CALLS_PATH) or not os.path.exists(CALLS_STAMP):
        return False
    with open(CALLS_STAMP) as f:
        if f.read() != _built_against():
            return False
    return all(os.path.getmtime(f) <= os.path.getmtime(CALLS_PATH)
               for f in (CALLS_SRC, os.path.join(ROOT, "include", "hca.h")))


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """The module behind the binding's paged calls (needs libhca.so)."""
    if not force and calls_up_to_date():
        return CALLS_PATH
    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = CALLS_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DHCA_TORCH_VERSION="{torch.__version__}"',
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(base, "include"),
           "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), CALLS_SRC, "-o", tmp, "-L" + PKG_DIR,
           "-l:" + os.path.basename(LIB_PATH), "-L" + os.path.join(base, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, CALLS_PATH)
    with open(CALLS_STAMP, "w") as f:
        f.write(_built_against())
    return CALLS_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    lib = _build_lib(force, verbose)
    build_calls(force, verbose)
    return lib


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + ".tmp"
    cmd = [_nvcc(), *NVCC_FLAGS, "-o", tmp, MAIN_SRC]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, verbose=True)
    print(path)
