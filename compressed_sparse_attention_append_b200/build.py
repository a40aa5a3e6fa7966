"""Builds libcsa2.so in-tree with nvcc for sm_100a (B200), and the binding's native marshalling (_marshal.so) with the
host compiler. Used by __graft_entry__.build()."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = [os.path.join(HERE, "csrc", f) for f in ("abi.cu", "append.cu", "index.cu", "index_decode.cu", "index_mma.cu", "attend.cu", "noalloc.cu", "latent.cu", "latent_index.cu",
                                         "rope.cu", "fp8.cu", "paged.cu", "layer_abi.cu")]
HDRS = [os.path.join(HERE, "csrc", "csa2_internal.cuh"), os.path.join(HERE, "csrc", "tc.cuh"), os.path.join(HERE, "csrc", "csa2_layer.cuh"),
        os.path.join(HERE, "csrc", "angle.cuh"), os.path.join(HERE, "csrc", "fp8_plan.h"),
        os.path.join(HERE, "csrc", "attend_plan.h"),
        os.path.join(ROOT, "include", "csa2.h"), os.path.join(ROOT, "include", "csa2_layer.h")]
LIB = os.path.join(HERE, "libcsa2.so")
MARSHAL_SRC = os.path.join(HERE, "csrc", "marshal.cpp")
MARSHAL = os.path.join(HERE, "_marshal.so")

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
    build_marshal(force)
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp, *SRC]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def build_marshal(force: bool = False) -> str:
    """The CPython module of csrc/marshal.cpp against the installed torch (8 s). layer.py works without it."""
    if not force and os.path.exists(MARSHAL) and all(os.path.getmtime(f) <= os.path.getmtime(MARSHAL) for f in (MARSHAL_SRC, HDRS[-1])):
        return MARSHAL
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    tmp = MARSHAL + f".tmp{os.getpid()}"
    inc = [*cpp_extension.include_paths(), "/usr/local/cuda/include", sysconfig.get_paths()["include"]]
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in inc), MARSHAL_SRC, "-o", tmp,
        *(f"-L{d}" for d in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, MARSHAL)
    return MARSHAL


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
