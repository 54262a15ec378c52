"""Build libqg.so in-tree: nvcc for sm_100a (CUDA sources) + the host packer, one shared object.

Usage: python -m quant_dequant_gemv_q4_b200.build [--force]
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libqg.so")
SOURCES = [os.path.join(CSRC, f) for f in ("qg_api.cu", "qg_heads.cu", "qg_attn.cu", "qg_sample.cu", "qg_pack.cpp")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cuh", ".h"))] \
    + [os.path.join(INCLUDE, "qg.h")]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_cmd(src: str, obj: str, extra=()) -> list[str]:
    return [NVCC, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, *extra,
            "-c", src, "-o", obj]


def build(force: bool = False, verbose: bool = False) -> str:
    """One object per source, compiled side by side, then linked."""
    stale = force or not os.path.exists(LIB) or any(
        os.path.getmtime(d) > os.path.getmtime(LIB) for d in DEPS)
    if stale:
        extra = ["-Xptxas", "-v"] if verbose else []
        objs = [f"{LIB}.{os.getpid()}.{os.path.basename(s)}.o" for s in SOURCES]
        tmp = LIB + f".tmp{os.getpid()}"
        try:
            with ThreadPoolExecutor(len(SOURCES)) as pool:
                list(pool.map(lambda so: subprocess.check_call(nvcc_cmd(*so, extra)), zip(SOURCES, objs)))
            subprocess.check_call([NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs])
            os.replace(tmp, LIB)
        finally:
            for o in objs:
                if os.path.exists(o):
                    os.remove(o)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
