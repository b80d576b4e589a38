"""Builds libnshb.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc.

Usage: python -m newton_schulz_hyperball_b200.build [--force]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libnshb.so")
SOURCES = ["api.cu", "stream_kernels.cu", "ns_f32.cu", "ns_tc2.cu", "himuon_tile.cu", "newton.cu", "newton_tc.cu",
           "norms_static.cu", "grad_norm.cu", "tensor_api.cu",
           "fp4.cu", "fp4_gemm.cu", "fp4_api.cu"]
HEADERS = ["nshb_internal.h", "nshb_device.cuh", "tensor_lists.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    for c in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libnshb.so")


def _inputs():
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "nshb.h")]
    return srcs, deps


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    _, deps = _inputs()
    return all(os.path.getmtime(d) <= t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    srcs, _ = _inputs()
    tmp = LIB + ".tmp"
    # --no-undefined: a symbol that no source defines fails the build instead of the first call
    cmd = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
           "-Xlinker", "--no-undefined", "-I", os.path.join(ROOT, "include"), "-o", tmp, *srcs]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
