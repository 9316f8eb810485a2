"""Build libds4a.so (the kernels and the C ABI) in-tree for sm_100a with nvcc.

    python -m long_context_hybrid_kv_b200.build [--force]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_lib", "libds4a.so")
BUILD = os.path.join(ROOT, "_build", "ds4a")

SOURCES = ["ds4a_api.cu", "ds4a_generic.cu", "ds4a_index_tc.cu", "ds4a_attend_tc.cu", "ds4a_noalloc.cu", "ds4a_topk.cu",
           "ds4a_selftest.cu", "ds4a_outproj.cu", "ds4a_mx.cu", "ds4a_paged.cu", "ds4a_paged_tc.cu", "ds4a_evict.cu", "ds4a_mxfp4.cu"]
HEADERS = ["ds4a_internal.cuh", "ds4a_tc.cuh", "ds4a_mx.cuh", "ds4a_paged.cuh", "ds4a_evict.cuh", "ds4a_mxfp4.cuh"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def _newer(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.exists(d) and os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "ds4a.h")]
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _newer(o, [s] + hdrs):
            cmd = [NVCC, *ARCH, *FLAGS, "-c", s, "-o", o]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}")
            log = os.path.join(BUILD, src.replace(".cu", ".ptxas.txt"))
            with open(log, "w") as f:
                f.write(r.stderr)
    if force or _newer(OUT, objs):
        cmd = [NVCC, *ARCH, "-shared", "-o", OUT, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
