"""Builds the sm_100a shared library libmoe_b200.so in-tree with nvcc, and the
native Python binding _moe_binding.<interpreter>.torch-<version>.so with g++.

    python -m expert_layer_dual_b200.build [--force]

Each .cu under csrc/ is compiled for sm_100a (-gencode arch=compute_100a,
code=sm_100a, -lineinfo) and linked into one shared library next to this
file, with the CUDA runtime linked statically.  Rebuilds only what is stale.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_b200.so")
SOURCES = ["api.cu", "routing.cu", "router.cu", "gemm_bf16.cu", "gemm_bf16_wide.cu", "gemm_bf16_2sm.cu", "gemm_fp8.cu", "gemm_mx.cu", "gemm_f8t.cu", "gemm_fp8_block.cu", "gemm_fp8_few.cu",
           "ep.cu", "allreduce_norm.cu", "noalloc.cu", "balance.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def binding_path() -> str:
    """The native binding for this interpreter and this torch: it is compiled against both,
    so its name says which, and another's is not found."""
    import torch
    return os.path.join(HERE, f"_moe_binding.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libmoe_b200.so")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(INCLUDE, "moe.h")]


def _mtime(p):
    return os.path.getmtime(p) if os.path.exists(p) else -1.0


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    path = os.path.join(CSRC, src)
    newest = max([_mtime(path)] + [_mtime(h) for h in _headers()])
    if _mtime(obj) < newest:
        cmd = [nvcc()] + ARCH + FLAGS + list(extra) + ["-c", path, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            if f.endswith(".o"):
                os.remove(os.path.join(BUILD, f))
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    if _mtime(LIB) < max(_mtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        if verbose:
            print("built", LIB)
    build_binding(force, verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The native argument marshalling (csrc/binding.cpp): a CPython module against
    this interpreter and its torch, linked to the library next to it."""
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    out = binding_path()
    newest = max(_mtime(src), _mtime(os.path.join(INCLUDE, "moe.h")))
    if force or _mtime(out) < newest:
        t = os.path.dirname(torch.__file__)
        tmp = out + f".tmp{os.getpid()}"
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-I", os.path.join(t, "include"),
               "-I", os.path.join(t, "include", "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], src, "-o", tmp, "-L", HERE, "-l:libmoe_b200.so",
               "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)
        if verbose:
            print("built", out)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
