"""Builds libtq.so (the CUDA library behind the C ABI in include/tq.h) and
_tq_torch.so (checks and marshalling of the short calls) in-tree.

    python kv_cache_vector_rope_b200/build.py          # compile if stale
    python kv_cache_vector_rope_b200/build.py --force  # always compile

Runs as a plain script (it must not import the package, whose binding loads
the library being built).

Everything is compiled for sm_100a only (B200).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtq.so")
BINDING_SRC = os.path.join(PKG, "binding", "tq_torch.cpp")
BINDING = os.path.join(PKG, "_tq_torch.so")
BINDING_FOR = os.path.join(PKG, "_tq_torch.for")      # the Python and torch that the binding was built for

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O3",
    "--expt-relaxed-constexpr",
    "-shared",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Both libraries, where they are stale; returns the path of libtq.so."""
    build_lib(force, verbose, extra)
    build_binding(force, verbose)
    return LIB


def build_lib(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *NVCC_FLAGS, *(extra or []), "-I", INCLUDE, "-I", CSRC, "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def _binding_stale(made_for: str) -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_FOR):
        return True
    with open(BINDING_FOR) as f:
        if f.read() != made_for:
            return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(p) > t for p in (BINDING_SRC, os.path.join(INCLUDE, "tq.h")))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The Python extension, by the host compiler against torch's headers; links libtq.so next to it. Its ABI is that of
    one Python and one torch: it is stale for others too."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    made_for = f"python {sysconfig.get_config_var('SOABI')}, torch {torch.__version__}\n"
    if not force and not _binding_stale(made_for):
        return BINDING
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include") if os.path.isabs(nvcc()) else None
    includes = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], INCLUDE, *([cuda] if cuda else [])]
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f for i in includes for f in ("-isystem", i)), "-o", tmp, BINDING_SRC, f"-L{PKG}", "-l:libtq.so",
           "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(made_for)
    return BINDING


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build_lib(force=force or bool(extra), verbose=True, extra=extra))
    print(build_binding(force=force, verbose=True))
