"""Builds libcsa2.so in-tree with nvcc for sm_100a (B200). Used by __graft_entry__.build()."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = [os.path.join(HERE, "csrc", f) for f in ("abi.cu", "append.cu", "index.cu", "index_decode.cu", "index_mma.cu", "attend.cu", "noalloc.cu", "latent.cu", "latent_index.cu",
                                         "rope.cu", "fp8.cu", "paged.cu", "layer_abi.cu")]
HDRS = [os.path.join(HERE, "csrc", "csa2_internal.cuh"), os.path.join(HERE, "csrc", "tc.cuh"), os.path.join(HERE, "csrc", "csa2_layer.cuh"),
        os.path.join(ROOT, "include", "csa2.h"), os.path.join(ROOT, "include", "csa2_layer.h")]
LIB = os.path.join(HERE, "libcsa2.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-shared",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in SRC + HDRS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp, *SRC]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
