"""Build libqg.so in-tree: nvcc for sm_100a (CUDA sources) + the host packer, one shared object; and, where torch is
installed, qg_binding.so, the Python side of the operators that take torch tensors.

Usage: python -m quant_dequant_gemv_q4_b200.build [--force]
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libqg.so")
BINDING = os.path.join(HERE, "qg_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "qg_binding.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("qg_api.cu", "qg_heads.cu", "qg_attn.cu", "qg_sample.cu", "qg_pack.cpp")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cuh", ".h"))] \
    + [os.path.join(INCLUDE, "qg.h")]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_cmd(src: str, obj: str, extra=()) -> list[str]:
    return [NVCC, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, *extra,
            "-c", src, "-o", obj]


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def built_for() -> str:
    """What a binding that is built now is built for: it is compiled against one torch and one Python."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = str(torch.__version__)
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}"


def binding_is_for(path: str) -> str | None:
    """What the binding at `path` was built for: noted beside it (and in it, for whoever loads it)."""
    try:
        with open(path + ".for") as f:
            return f.read()
    except OSError:
        return None


def build_binding(force: bool = False) -> str:
    """Needs torch, its headers and Python's."""
    deps = [BINDING_SOURCE, os.path.join(INCLUDE, "qg.h")]
    if force or not os.path.exists(BINDING) or binding_is_for(BINDING) != built_for() or any(
            os.path.getmtime(d) > os.path.getmtime(BINDING) for d in deps):
        import torch
        root = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(NVCC))
        paths = [x for p in (f"{root}/include", f"{root}/include/torch/csrc/api/include", f"{cuda}/include") for x in ("-isystem", p)]
        tmp = BINDING + f".tmp{os.getpid()}"
        try:
            subprocess.check_call(["g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-fvisibility=hidden",
                                   f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                                   f'-DQG_BUILT_FOR="{built_for()}"', "-I", INCLUDE,
                                   "-I", sysconfig.get_paths()["include"], *paths, BINDING_SOURCE, "-o", tmp, "-L", f"{root}/lib",
                                   "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
            os.replace(tmp, BINDING)
            with open(BINDING + ".for", "w") as f:
                f.write(built_for())
        finally:
            if os.path.exists(tmp):
                os.remove(tmp)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """One object per source, compiled side by side, then linked; then the binding, which libqg.so does without."""
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
    if has_torch():
        build_binding(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
