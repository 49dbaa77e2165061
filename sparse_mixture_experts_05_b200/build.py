"""Build libmoe.so (the sm_100a CUDA kernels and the C ABI) in-tree with nvcc.

    python -m sparse_mixture_experts_05_b200.build [--force] [--verbose-ptxas]

Objects go to _build/ at the repository root; the shared library lands next to
this file so that it travels with the package.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe.so")
SOURCES = ["api.cu", "router.cu", "dispatch.cu", "expert_gemm.cu", "combine.cu", "aux_loss.cu",
           "tma_map.cu", "api_int8.cu", "route_scored.cu", "route_scored_bf16.cu",
           "int8_rows.cu", "expert_int8.cu"]
HEADERS = ["common.cuh", "sm100.cuh", "expert_gemm.cuh", "router.cuh", "dispatch.cuh",
           "combine.cuh", "combine_math.cuh", "aux_loss.cuh", "tma_map.cuh", "route_scored.cuh",
           "route_scored_kernels.cuh", "int8_rows.cuh", "expert_int8.cuh"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "moe.h")]
    objs, cmds = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or verbose_ptxas or _stale(o, [s] + hdrs):
            cmd = [NVCC, *ARCH, *FLAGS, "-c", s, "-o", o]
            if verbose_ptxas:
                cmd.insert(1, "-Xptxas=-v")
            cmds.append(cmd)
    with ThreadPoolExecutor(os.cpu_count() or 1) as pool:  # one nvcc a source, side by side
        list(pool.map(subprocess.check_call, cmds))
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        subprocess.check_call([NVCC, *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp])
        os.replace(tmp, LIB)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
    return 0


if __name__ == "__main__":
    sys.exit(main())
