"""Builds libcsa2.so in-tree with nvcc for sm_100a (B200), and the binding's native marshalling (_marshal.so) with the
host compiler. Used by __graft_entry__.build()."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings

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
# (named for the interpreter it is built against: another one does not find it)
MARSHAL = os.path.join(HERE, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

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
    """The library, and the marshalling where it can be built (without Python's or torch's headers it cannot, and the
    library alone is what a C program needs)."""
    if force or stale():
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([_nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp, *SRC])
        os.replace(tmp, LIB)
    try:
        build_marshal(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the binding's native marshalling is not built ({e}); its Python code makes every call")
    return LIB


def _marshal_stale(abi: str) -> bool:
    try:
        with open(MARSHAL + ".abi") as f:
            if f.read() != abi:
                return True
        t = os.path.getmtime(MARSHAL)
    except OSError:
        return True
    return any(os.path.getmtime(f) > t for f in (MARSHAL_SRC, HDRS[-1], HDRS[-2]))


def build_marshal(force: bool = False) -> str:
    """The CPython module of csrc/marshal.cpp against the installed torch (8 s). layer.py works without it. What was built
    against another torch, or from older sources, does not stay, whether or not the new build succeeds."""
    import torch

    abi = f"{sys.implementation.cache_tag} torch {torch.__version__} cxx11 {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    if not force and not _marshal_stale(abi):
        return MARSHAL
    for old in (MARSHAL, MARSHAL + ".abi", os.path.join(HERE, "_marshal.so")):
        if os.path.exists(old):
            os.remove(old)
    from torch.utils import cpp_extension

    tmp = MARSHAL + f".tmp{os.getpid()}"
    inc = [*cpp_extension.include_paths(), "/usr/local/cuda/include", sysconfig.get_paths()["include"]]
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in inc), MARSHAL_SRC, "-o", tmp,
        *(f"-L{d}" for d in cpp_extension.library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, MARSHAL)
    with open(MARSHAL + ".abi", "w") as f:
        f.write(abi)
    return MARSHAL


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
