"""Build step: compile the CUDA library into moe_grouped_gemm_fp32_b200/_dg.so.

nvcc cross-compiles for sm_100a only (no other architecture is generated);
the CUDA runtime is linked statically and the driver's tensor-map encoder is
fetched at run time, so the library needs no -lcuda.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("dg_api.cu", "quant_api.cu", "bf16_api.cu",
                                              "ragged_api.cu", "w4_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("gemm_kernel.cuh", "ptx.cuh", "quant_kernel.cuh",
                                                  "bf16_kernel.cuh", "ragged_kernel.cuh", "w4_kernel.cuh", "pdl.cuh",
                                                  "api_common.h")] + [
    os.path.join(ROOT, "include", "dg.h")]
OUT = os.path.join(HERE, "_dg.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(f) <= t for f in DEPS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return OUT
    tmp = OUT + f".tmp{os.getpid()}"
    cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-o", tmp] + SOURCES
    subprocess.check_call(cmd)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(OUT)
