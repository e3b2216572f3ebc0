"""Build librmsmod.so (sm_103a) in-tree with nvcc; no CMake, one -gencode.

Each translation unit is compiled in parallel, then linked into a shared
library with the CUDA runtime linked statically.  Rebuilds only when a
source or the public header is newer than the library.
"""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librmsmod.so")
HEADER = os.path.join(ROOT, "include", "rmsmod.h")

SOURCES = ["api.cu", "row_kernels.cu", "qk_kernel.cu", "wan_kernel.cu", "elementwise.cu",
           "backward.cu", "mxfp4.cu", "mxfp4_matmul.cu", "mxfp8.cu", "mxfp8_matmul.cu",
           "mxfp8_norm.cu", "sandwich.cu",
           "selftest.cu"]

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = [
    *ARCH, "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    # no contraction of separate fp32 multiply/add, IEEE divide/sqrt, no FTZ:
    # rounding-sensitive steps are explicit .rn instructions anyway
    "-fmad=false", "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
]


def _deps():
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return paths + [HEADER, os.path.abspath(__file__)]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [NVCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr:
        print(res.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
