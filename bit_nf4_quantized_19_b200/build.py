"""Build libqlora_nf4.so in-tree for sm_100a with nvcc (no JIT cache).

    python -m bit_nf4_quantized_19_b200.build [--ptxas-verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libqlora_nf4.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

SOURCES = ["qlora_nf4.cu", "nf4_table.cpp"]
HEADERS = ["adapter_mma.cuh", "common.cuh", "fp8_gemm.cuh", "fp8_layer.cuh", "fp8_quant.cuh", "fp8_skinny.cuh",
           "gemm_kernel.cuh", "lora_mma.cuh", "merge_kernel.cuh", "pipeline.cuh", "quant_kernels.cuh",
           "skinny_kernel.cuh", "nf4_table.hpp", "workspace.hpp"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "-shared",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "qlora_nf4.h")]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    """Compile the library if any source is newer than the .so; return its path."""
    if not force and not _stale():
        return LIB_PATH
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB_PATH + ".tmp"
    cmd += ["-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if not quiet or ptxas_verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    v = "--ptxas-verbose" in sys.argv
    print(build(force=True, ptxas_verbose=v, quiet=False))
