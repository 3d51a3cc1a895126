"""Build libtb.so in-tree with nvcc for sm_100a, and _tbcall.so (the Python
side's argument marshalling, host code only) with g++.

    python -m query_aware_sparse_tb_b200.build

Objects go to query_aware_sparse_tb_b200/_build/, the shared library to
query_aware_sparse_tb_b200/libtb.so.  No GPU is needed (nvcc cross-compiles).
libtb.so needs nvcc alone.  Where _tbcall.so cannot be built (no g++, no torch or
Python headers), build() warns: the C ABI and the ctypes calls work without it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

from ._lib import call_tag

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtb.so")
CALL = os.path.join(PKG, "_tbcall.so")
SOURCES = ["api.cu", "attn.cu", "select.cu", "select_cluster.cu", "gemm_tc.cu", "noalloc.cu", "kv.cu",
           "multi_attn.cu", "rope.cu", "tree.cu"]
NVCC = os.environ.get("NVCC", "nvcc")
CXX = "g++"  # the system's, whose C++ runtime torch shares: exceptions cross between the two
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-cudart", "shared", "-I", os.path.join(ROOT, "include")]


def _newer(out: str, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(out) >= os.path.getmtime(d) for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "tb.h"))
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or not _newer(o, [s] + headers):
            jobs.append([NVCC, *FLAGS, "-c", s, "-o", o])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for cmd, res in zip(jobs, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs)):
                if res.returncode != 0:
                    raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
                if verbose and res.stderr.strip():
                    print(res.stderr, file=sys.stderr)
    if force or jobs or not _newer(LIB, objs):
        cmd = [NVCC, "-shared", "-cudart", "shared", "-gencode", "arch=compute_100a,code=sm_100a",
               "-o", LIB, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    try:
        build_call(force)
    except (OSError, ImportError, RuntimeError) as e:
        warnings.warn(f"libtb.so is built, _tbcall.so is not (norm_rope_append, prompt_attn, tree_attn and tree_accept "
                      f"need it from Python): {e}")
    return LIB


def build_call(force: bool = False) -> str:
    """_tbcall.so: a CPython module over torch's C++ headers, built again when
    its sources, torch or Python are others than it was built for."""
    src, stamp = os.path.join(CSRC, "tbcall.cpp"), os.path.join(BUILD, "_tbcall.tag")
    tag, built = call_tag(), None
    if os.path.exists(stamp):
        with open(stamp) as f:
            built = f.read()
    if force or built != tag or not _newer(CALL, [src, os.path.join(ROOT, "include", "tb.h")]):
        import sysconfig

        import torch
        base = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or "/usr/local/cuda/bin/nvcc")))
        tmp = f"{CALL}.{os.getpid()}.tmp"
        cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f'-DTB_BUILT_FOR="{tag}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-isystem", os.path.join(base, "include"),
               "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
               "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
               src, "-o", tmp, "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
               f"-Wl,-rpath,{os.path.join(base, 'lib')}"]
        try:
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"{CXX} failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        except (OSError, RuntimeError):
            if os.path.exists(CALL):  # it does not belong to these sources
                os.remove(CALL)
            raise
        os.replace(tmp, CALL)
        os.makedirs(BUILD, exist_ok=True)
        with open(stamp, "w") as f:
            f.write(tag)
    return CALL


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
