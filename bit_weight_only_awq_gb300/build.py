"""Builds libawq.so in-tree with nvcc for sm_103a (one -gencode, parallel translation units).

Usage: ``python -m bit_weight_only_awq_gb300.build`` (also called by ``__graft_entry__.build``).
Objects go to ``_build/`` at the repository root; the shared library lands next to this file.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libawq.so")

SOURCES = ("awq_api.cu", "awq_elementwise.cu", "awq_gemv.cu", "awq_gemv_pp.cu", "awq_gemm_tc.cu", "w4a8_act.cu",
           "awq_noalloc.cu", "awq_selftest.cu", "w4a8_rmsnorm.cu", "kv4_cache.cu", "kv4_attention.cu",
           "kv4_prefill.cu", "moe_route.cu", "moe_pack.cu", "moe_gemm.cu", "fp8_quant.cu", "fp8_gemm.cu")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libawq.so")


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    return obj


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    """Compile every translation unit and link libawq.so; returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs_mtime = max(os.path.getmtime(os.path.join(CSRC, s)) for s in SOURCES)
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hdrs.append(os.path.join(ROOT, "include", "awq.h"))
    srcs_mtime = max([srcs_mtime] + [os.path.getmtime(h) for h in hdrs])
    if not force and os.path.exists(LIB_PATH) and os.path.getmtime(LIB_PATH) >= srcs_mtime:
        return LIB_PATH
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv, force="-f" in sys.argv))
