"""Build ``libsbl.so`` (the sm_100a CUDA library behind include/sbl.h) in-tree.

    python -m sparsity_sbl_quantize_b200.build [--force] [--verbose]

nvcc cross-compiles for sm_100a without a GPU.  The library is three
translation units -- csrc/sbl_api.cu (the ABI of the ternary layer; it
includes its kernel headers), csrc/sbl_b8_api.cu (the 8-bit block operators)
and csrc/sbl_container.cpp (the host-only packed-layer container), compiled
side by side -- linked against the static CUDA runtime; the driver entry point for tensor-map encoding is
looked up at run time, so libcuda is not a link dependency.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsbl.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills", "--threads", "0",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "sbl.h")])


def build(force: bool = False, verbose: bool = False) -> str:
    newest = max(os.path.getmtime(p) for p in sources())
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return LIB
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", tmp,
           os.path.join(CSRC, "sbl_api.cu"), os.path.join(CSRC, "sbl_b8_api.cu"),
           os.path.join(CSRC, "sbl_container.cpp")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
