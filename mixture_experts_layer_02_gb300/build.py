"""In-tree build of libmoe.so (hand-written CUDA for sm_103a).

    python -m mixture_experts_layer_02_gb300.build [--force] [--ptxas-verbose]

Each translation unit compiles in parallel with nvcc for exactly one target,
``-gencode arch=compute_103a,code=sm_103a``; objects go to ``_build/`` and the
shared library is linked next to this file, where the binding loads it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
SOURCES = ["grouped_gemm.cu", "grouped_gemm_e4m3.cu", "grouped_gemm_2sm.cu", "grouped_gemm_2sm_e4m3.cu",
           "grouped_gemm_2sm_mixed.cu",
           "grouped_gemm_swap.cu", "grouped_gemm_swap_e4m3.cu", "grouped_gemm_gather.cu",
           "grouped_gemm_gather_e4m3.cu", "grouped_gemm_gather_small.cu", "ffn_fused_decode.cu", "layer_decode.cu", "quant.cu", "route_reduce.cu",
           "permute.cu", "combine.cu", "rmsnorm.cu", "dense_grad.cu", "dense_gemm_split_gated.cu",
           "dense_gemm_split_linear.cu", "dense_gemm_split_dgrad.cu", "dense_gemm_split_wgrad.cu",
           "dense_gemm_pairsplit_gated.cu", "dense_gemm_pairsplit_linear.cu", "dense_gemm_pairsplit_dgrad.cu",
           "dense_gemm_pairsplit_wgrad.cu",
           "dense_gemm_pair.cu", "dense_gemv.cu", "dense_api.cu",
           "moe_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmoe.so")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "moe.h")]


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = _headers()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include")]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or ptxas_verbose or _newer(o, [s] + hdrs):
            cmd = [nvcc()] + flags + ["-c", s, "-o", o + ".tmp"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            os.replace(o + ".tmp", o)
            if ptxas_verbose or not quiet:
                sys.stderr.write(r.stderr)
        return o

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    if force or _newer(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose, quiet=False))
