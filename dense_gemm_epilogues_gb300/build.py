"""Build libgemm.so (in-tree) with nvcc for sm_103a.

The translation units are compiled in parallel and linked into
``dense_gemm_epilogues_gb300/libgemm.so``; objects go to ``_build/``.  The
CUDA runtime is linked statically, the driver API (TMA descriptor encoding) is
reached through the runtime's driver entry-point query, so the library has no
link-time dependency on libcuda.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgemm.so")
SOURCES = ["gemm_api.cu", "tc_kernel.cu", "tc2_kernel.cu", "simt_kernels.cu", "diag_kernel.cu",
           "pair_kernel.cu", "expert_api.cu", "q4_kernel.cu", "repitch_kernel.cu", "ortho_kernels.cu", "seg_kernel.cu",
           "layer_api.cu", "linear_kernel.cu", "route_kernels.cu", "exchange_kernels.cu", "clip_kernels.cu"]
HEADERS = ["common.cuh", "kernels.h", "plan.h", "activation.cuh", "expert.h", "operands.h", "layer.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(PKG, "..", "include", "gemm.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _inputs_mtime():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]
    # Extra nvcc flags for tuning builds (e.g. -DGEMM_PAIR_STAGES=7); pass force=True to rebuild.
    flags += os.environ.get("GEMM_EXTRA_NVCC_FLAGS", "").split()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc()] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
