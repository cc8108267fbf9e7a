"""A block whose wait runs out still waits for its own copies and MMAs in flight before it gives up its
shared memory and TMEM, and that last wait does not shrink with the caller's limit.  Read from
the sources: making a wait run out in a kernel at work is left to the reader."""
import os
import re

import pytest

from bit_nf4_quantized_19_b200 import build

KERNEL = re.compile(r"__global__.*?(?=__global__|\n}  // namespace)", re.S)
FINAL = re.compile(r"Waiter \w+\{&no_abort, (.*)\};")


def kernels():
    """(name, text) of each kernel that loads by TMA or the bulk-copy engine; the body of lora_mma_kernel is a
    device function in front of it."""
    out = []
    for name in sorted(build.HEADERS):
        text = re.sub(r"//(?! namespace)[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
        if name == "lora_mma.cuh":
            out.append(("lora_mma_kernel", text))
            continue
        out += [(re.search(r"(\w+_kernel)\s*\(", m.group(0)).group(1), m.group(0)) for m in KERNEL.finditer(text)
                if re.search(r"\b(tma_load_\dd\w*|bulk_load)\(", m.group(0))]
    return out


def test_the_kernels_are_found():
    assert sorted(n for n, _ in kernels()) == [
        "adapter_mma_kernel", "fp8_gemm_kernel", "fp8_skinny_kernel", "lora_mma_kernel", "nf4_merge_kernel",
        "nf4_quantize_kernel", "qlora_gemm_kernel", "qlora_skinny_kernel", "qlora_xa_kernel"]


@pytest.mark.parametrize("name,text", kernels(), ids=[n for n, _ in kernels()])
def test_the_last_waits_have_their_own_limit(name, text):
    limits = FINAL.findall(text)
    if not limits:      # no phase to wait on, or no registers for it: a fixed delay, long against a copy's time
        assert re.search(r"if \(!ok\) \{\s*(#pragma unroll 1\s*)?for \(int i = 0; i < 200; \+\+i\) __nanosleep\(1000\);", text)
        return
    assert all(x == "p.drain_ns" or x.startswith("drain_limit_ns(") for x in limits)


def test_limits_from_the_host():
    """Each struct with a drain_ns is filled from drain_limit_ns by its one launch."""
    structs = sum(len(re.findall(r"uint64_t drain_ns;", open(os.path.join(build.CSRC, n)).read())) for n in build.HEADERS)
    host = open(os.path.join(build.CSRC, "qlora_nf4.cu")).read()
    assert structs == len(re.findall(r"p\.limit_ns = [^\n]*\n  p\.drain_ns = drain_limit_ns\(p\.limit_ns\);", host)) == 3


@pytest.mark.parametrize("name,text", [k for k in kernels() if "mma_commit" in k[1]],
                         ids=[n for n, t in kernels() if "mma_commit" in t])
def test_every_mma_is_waited_for(name, text):
    """A commit behind the issuer's loop, whichever way it was left, and a last wait for it."""
    bar = re.findall(r"(?:mma_commit(?:_pair)?|commit)\((drain|done)\b", text)
    assert bar
    assert re.search(r"wait_bar(?:_warp)?\(%s, 0, (?:final_wt|dw)\)" % bar[0], text)
