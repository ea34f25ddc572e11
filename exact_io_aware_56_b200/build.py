"""Builds libfa.so and its torch binding in-tree with nvcc for sm_100a.

Usage: ``python -m exact_io_aware_56_b200.build`` (or ``build()`` from
Python). The library is written next to this file so that it travels with
the source tree; nothing is installed elsewhere.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libfa.so")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_bwd_noalloc.cu", "fa_decode.cu", "fa_quant.cu", "fa_packed.cu",
           "fa_paged.cu", "fa_rope.cu"]
# The native binding of the packed, paged and rotary calls: a Python module that links libfa.so.
BINDING = os.path.join(HERE, "_fa_torch.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa.so")


def build_binding() -> str:
    """Compiles the torch binding (host code only) against libfa.so; returns its path."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    incs = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    libs = library_paths()
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-isystem{i}" for i in incs],
           os.path.join(CSRC, "torch_binding.cpp"), "-o", BINDING + ".tmp", LIB, "-Wl,-rpath,$ORIGIN",
           *[f"-L{d}" for d in libs], "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(verbose: bool = False, extra=None) -> str:
    """Compiles every CUDA source into libfa.so, then the torch binding; returns libfa.so's path."""
    cmd = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
           "-Xcompiler", "-fPIC", "-shared", "-Xlinker", "-soname=libfa.so", "-I", os.path.join(ROOT, "include"),
           "-o", LIB + ".tmp", *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    if extra:
        cmd[1:1] = list(extra)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    os.replace(LIB + ".tmp", LIB)
    build_binding()
    if verbose:
        sys.stdout.write(res.stdout + res.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
