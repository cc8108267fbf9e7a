"""Arguments that are refused before anything is launched.  No call reaches a GPU."""
import ctypes

import pytest
import torch

import bit_nf4_quantized_19_b200 as q
from bit_nf4_quantized_19_b200 import _abi, build


@pytest.mark.parametrize("given", [(), ("dA",), ("dB",)])
def test_accumulate_needs_both_gradients(given):
    """Without both there is nothing to add into: linear_bwd made them up from unwritten memory."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    g = {k: torch.zeros(128, 128) for k in given}
    with pytest.raises(ValueError):
        q.linear_bwd(x, x, None, None, x, x, 1.0, accumulate=True, **g)


# ------------------------------------------------------------------ results over operands
M, N, K, R = 8, 256, 256, 8
BASE = 1 << 20                        # addresses only: every call below is refused


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


def p(a):
    return ctypes.c_void_p(a)


def calls(L, out, act, saved):
    """The C calls whose bf16 result `out` has the shape of a bf16 operand `act` (and, of the NF4 backward, `saved`),
    with a workspace of no bytes: what passes the checks of arguments ends there (or, without a GPU, before)."""
    w4 = ctypes.byref(_abi.NF4Struct(64 << 20, 65 << 20, 66 << 20, N, K))
    x8 = ctypes.byref(_abi.FP8Struct(67 << 20, 68 << 20, M, K, 0, 1))
    w8 = ctypes.byref(_abi.FP8Struct(69 << 20, 70 << 20, N, K, 0, 128))
    A, B, dA, dB, ws = p(71 << 20), p(72 << 20), p(73 << 20), p(74 << 20), p(75 << 20)
    return dict(
        linear_fwd=L.qlora_linear_fwd(p(act), M, w4, A, B, R, 1.0, p(out), None, ws, 0, None),
        linear_bwd=L.qlora_linear_bwd(p(act), p(saved), None, M, w4, A, B, R, 1.0, p(out), dA, dB, ws, 0, None),
        linear_bwd_ckpt=L.qlora_linear_bwd_ckpt(p(act), x8, None, w4, A, B, R, 1.0, None, 0.0, 0, p(out), dA, dB, ws, 0, None),
        fp8_linear_bwd=L.qlora_fp8_linear_bwd(p(act), M, x8, None, w8, A, B, R, 1.0, 0, 0, p(out), dA, dB, ws, 0, None),
        fp8_product_bwd=L.qlora_fp8_linear_bwd(p(act), M, None, None, w8, None, None, 0, 1.0, 0, 0, p(out), None, None, ws, 0,
                                               None))


BYTES = 2 * M * K


@pytest.mark.parametrize("shift", [0, 16, -16, BYTES - 16, 16 - BYTES])
def test_a_result_over_an_operand_is_refused(L, shift):
    """Tiles of the result are written while others of the operand are still to be read."""
    assert set(calls(L, BASE + shift, BASE, 80 << 20).values()) == {1}
    assert calls(L, BASE + shift, 80 << 20, BASE)["linear_bwd"] == 1


@pytest.mark.parametrize("shift", [BYTES, -BYTES])
def test_a_result_beside_an_operand_is_not(L, shift):
    assert set(calls(L, BASE + shift, BASE, 80 << 20).values()) <= {7, 8}     # no workspace, or no GPU
    assert calls(L, BASE + shift, 80 << 20, BASE)["linear_bwd"] in (7, 8)
