"""Build libvitq.so in-tree with nvcc for sm_100a (no JIT cache, no torch extension)."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libvitq.so")
SOURCES = ["vitq_all.cu", "elementwise.cu", "gemm_fp8.cu", "gemm_bf16.cu", "attention.cu", "api.cu", "merger_static.cu",
           "quant_int8.cu", "gemm_int8.cu", "rope_axes.cu", "int8_api.cu", "ptx.cuh", "internal.h",
           "int8_choose.h"]


def nvcc_cmd(out: str = LIB, extra=()) -> list:
    return ["nvcc", "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
            "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
            *extra, "-o", out, os.path.join(CSRC, "vitq_all.cu")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(ROOT, "include", "vitq.h")]
    return all(os.path.getmtime(d) <= t for d in deps)


def build(force: bool = False, verbose: bool = True) -> str:
    if not force and up_to_date():
        return LIB
    cmd = nvcc_cmd()
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv)
