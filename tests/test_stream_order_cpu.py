"""Kernels that start before the kernel in front of them has ended (they call griddepcontrol.wait) read
global memory by coherent loads only: the non-coherent path (ld.global.nc, __ldg, const __restrict__)
is for memory that nobody writes while the grid lives, and the kernel in front may still be
writing when the grid begins.  Read from the sources."""
import os
import re

import pytest

from bit_nf4_quantized_19_b200 import build

KERNEL = re.compile(r"__global__.*?(?=__global__|\n}  // namespace)", re.S)
WAITS = re.compile(r"\bpdl_wait\(\)|griddepcontrol\.wait")
NONCOHERENT = re.compile(r"__ldg\w*\(|ld_global_nc\w*\(|\.nc\b|__restrict__")


def kernels():
    """(file, text from __global__ on, comments taken out) of each kernel that waits for another."""
    out = []
    for name in sorted(build.HEADERS + build.SOURCES):
        text = open(os.path.join(build.CSRC, name)).read()
        text = re.sub(r"//(?! namespace)[^\n]*", "", text)
        out += [(name, m.group(0)) for m in KERNEL.finditer(text) if WAITS.search(m.group(0))]
    return out


@pytest.mark.parametrize("name,text", kernels(), ids=lambda v: v if len(v) < 40 else re.search(r"(\w+_kernel)\(", v).group(1))
def test_no_non_coherent_load_behind_a_wait(name, text):
    assert not NONCOHERENT.findall(text)


def test_the_kernels_are_found():
    found = {re.search(r"(\w+_kernel)\(", t).group(1) for _, t in kernels()}
    assert found == {"adapter_mma_kernel", "fp8_gemm_kernel", "fp8_reduce_kernel", "fp8_quantize_kernel", "fp8_skinny_kernel",
                     "qlora_skinny_kernel", "qlora_xa_kernel"}
