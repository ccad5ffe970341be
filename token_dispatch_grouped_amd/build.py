"""Build the HIP library ``libmoe_mi355x.so`` in-tree for gfx950.

Usage: ``python -m token_dispatch_grouped_amd.build`` (or ``build()`` from
Python). Every source is compiled with hipcc for gfx950 only; packed-fp32
instructions are disabled for the device code. Objects go to ``_build/``
next to this file; the shared library lands next to this file.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libmoe_mi355x.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)

SOURCES = ["moe_abi.cpp", "validate.cpp", "route.hip", "dispatch.hip", "gemm_bf16.hip", "gemm_bf16_ilp.hip",
           "gemm_f32.hip", "optim.hip", "aux.hip", "peak.hip", "ep.hip", "norm.hip", "ffn.hip", "ffn_ilp.hip"]
# Per-source compiler options: the gate/up forward and weight-gradient GEMM
# kernels (gemm_bf16_ilp.hip) are scheduled for instruction-level parallelism,
# which makes them 0.5-1.8% faster and the dgrad kernels slower (those are in
# gemm_bf16.hip, default scheduler).
SOURCE_FLAGS = {"gemm_bf16_ilp.hip": ["-mllvm", "--amdgpu-sched-strategy=max-ilp"],
                "ffn_ilp.hip": ["-mllvm", "--amdgpu-sched-strategy=max-ilp"]}
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found; the ROCm toolchain is required to build the MoE library")


def common_flags():
    return ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wno-unused-command-line-argument"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [hipcc()] + common_flags() + SOURCE_FLAGS.get(src, []) + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    """Compile every source and link the shared library. Always rebuilds."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp"
    # roctx: named ranges around the C-ABI calls for marker traces
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs + [
        "-L/opt/rocm/lib", "-lrocprofiler-sdk-roctx", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build()
    sys.exit(0)
