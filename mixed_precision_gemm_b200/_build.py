"""Build of the CUDA library (libsq_b200.so) for sm_100a, in the package folder.

nvcc cross-compiles without a GPU, so this runs on any machine with CUDA 12.8+.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_NAME = "libsq_b200.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["sq_abi.cu"]
DEPS = ["sq_abi.cu", "sq_device.cuh", "sq_fp8b.cuh", "sq_fp8b_host.cuh", "sq_fp8b_pair.cuh", "sq_fp8b_skinny.cuh", "sq_gemm_common.cuh", "sq_gemm_pair.cuh", "sq_gemm_skinny.cuh", "sq_moe.cuh", "sq_mxquant.cuh", "sq_rowquant.cuh", "sq_rowquant_stream.cuh", "sq_select.cuh", "sq_sqf.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=true",
    "-Xcompiler", "-fPIC", "-shared",
    "-I", os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    paths = [os.path.join(CSRC, d) for d in DEPS] + [os.path.join(ROOT, "include", "sq.h")]
    return any(os.path.getmtime(p) > t for p in paths)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile the library if it is missing or older than its sources."""
    if not (force or _stale()):
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(extra_flags or []),
           *[os.path.join(CSRC, s) for s in SOURCES], "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
