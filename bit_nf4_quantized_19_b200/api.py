"""Tensor-level wrappers over the C ABI (PyTorch supplies device memory and streams).

Each function allocates its outputs with torch, passes raw device pointers and
the current CUDA stream to libqlora_nf4.so and returns the tensors.  No
arithmetic of the method happens here.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Tuple

import torch

from . import _abi


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _bf16_2d(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_cuda:
        raise TypeError(f"{name} must be a 2-D bfloat16 CUDA tensor")
    return t.contiguous()


@dataclasses.dataclass
class NF4Weight:
    """A quantized frozen weight [rows, cols]: packed codes, 8-bit block
    constants, fp32 group constants (device tensors owned by this object).  With
    q8 = None the constants are single-level: `step` holds one fp32 absmax per
    64-value block."""
    codes: torch.Tensor
    q8: Optional[torch.Tensor]
    step: torch.Tensor
    rows: int
    cols: int

    def c_struct(self) -> _abi.NF4Struct:
        return _abi.NF4Struct(self.codes.data_ptr(), self.q8.data_ptr() if self.q8 is not None else None,
                              self.step.data_ptr(), self.rows, self.cols)

    @property
    def single_level(self) -> bool:
        return self.q8 is None

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + (self.q8.numel() if self.q8 is not None else 0) + 4 * self.step.numel()


_FP8_FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@dataclasses.dataclass
class FP8Tensor:
    """A matrix in blockwise 8-bit floating point (device tensors owned by this object):
    codes [rows, cols] in float8_e4m3fn or float8_e5m2, and one power-of-two byte e + 127
    per block of block_rows x 128 values, scales uint8 [ceil(rows / block_rows),
    4 ceil(cols / 512)].  block_rows is 1 for activations and gradients (the 8-bit
    activation checkpoint), 128 for a weight [N, K]."""
    codes: torch.Tensor
    scales: torch.Tensor
    block_rows: int = 1

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def cols(self) -> int:
        return self.codes.shape[1]

    @property
    def fmt(self) -> str:
        return "e5m2" if self.codes.dtype == torch.float8_e5m2 else "e4m3"

    @property
    def device(self) -> torch.device:
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def check(self, name: str, block_rows: Optional[int] = None) -> Tuple[int, int]:
        """(rows, cols); raises unless the two tensors are what the library reads."""
        c, s, br = self.codes, self.scales, self.block_rows
        if (c.dtype != torch.float8_e4m3fn and c.dtype != torch.float8_e5m2) or c.dim() != 2 or not c.is_cuda:
            raise TypeError(f"{name}.codes must be a 2-D float8_e4m3fn or float8_e5m2 CUDA tensor")
        if s.dtype != torch.uint8 or s.device != c.device:
            raise TypeError(f"{name}.scales must be a uint8 tensor on the device of the codes")
        if br not in (1, 128) or (block_rows is not None and br != block_rows):
            raise ValueError(f"{name}.block_rows is {br}, expected {block_rows or '1 or 128'}")
        if br == 128 and c.dtype != torch.float8_e4m3fn:
            raise TypeError(f"{name}: 128 x 128 blocks are e4m3")
        rows, cols = c.shape
        if s.shape != _fp8_scale_shape(rows, cols, br) or not c.is_contiguous() or not s.is_contiguous():
            raise ValueError(f"{name} must be contiguous with scales {_fp8_scale_shape(rows, cols, br)}, "
                             f"got {tuple(s.shape)}")
        return rows, cols

    def c_struct(self) -> bytes:
        """The library's view of this tensor (qlora_fp8_t)."""
        c = self.codes
        rows, cols = c.shape
        return _abi.pack_fp8(c.data_ptr(), self.scales.data_ptr(), rows, cols,
                             1 if c.dtype == torch.float8_e5m2 else 0, self.block_rows)


def _fp8_scale_shape(rows: int, cols: int, block_rows: int) -> Tuple[int, int]:
    return (rows + block_rows - 1) // block_rows, 4 * ((cols + 511) // 512)


def nf4_levels() -> list:
    buf = (ctypes.c_float * 16)()
    _abi.lib().qlora_nf4_levels(buf)
    return list(buf)


def nf4_bytes(rows: int, cols: int) -> Tuple[int, int, int]:
    c, q, s = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _abi.lib().qlora_nf4_bytes(rows, cols, ctypes.byref(c), ctypes.byref(q), ctypes.byref(s))
    return c.value, q.value, s.value


def nf4_empty(rows: int, cols: int, device) -> NF4Weight:
    cb, qb, sb = nf4_bytes(rows, cols)
    return NF4Weight(torch.empty(cb, dtype=torch.uint8, device=device),
                     torch.empty(qb, dtype=torch.uint8, device=device),
                     torch.empty(sb // 4, dtype=torch.float32, device=device), rows, cols)


def nf4_empty_single(rows: int, cols: int, device) -> NF4Weight:
    """Storage for single-level constants (one fp32 absmax per 64-value block)."""
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    _abi.lib().qlora_nf4_single_bytes(rows, cols, ctypes.byref(c), ctypes.byref(s))
    return NF4Weight(torch.empty(c.value, dtype=torch.uint8, device=device), None,
                     torch.empty(s.value // 4, dtype=torch.float32, device=device), rows, cols)


def nf4_quantize(W: torch.Tensor, out: Optional[NF4Weight] = None, single_level: bool = False) -> NF4Weight:
    """Blockwise NF4 quantization of a bf16 [rows, cols] CUDA tensor, with
    double-quantized constants (default) or single-level fp32 ones."""
    W = _bf16_2d(W, "W")
    rows, cols = W.shape
    if out is not None:
        q = out
    else:
        q = nf4_empty_single(rows, cols, W.device) if single_level else nf4_empty(rows, cols, W.device)
    st = q.c_struct()
    _abi.check(_abi.lib().qlora_nf4_quantize(_ptr(W), rows, cols, ctypes.byref(st),
                                             _stream(W.device)), "qlora_nf4_quantize")
    return q


def nf4_dequant(Wq: NF4Weight, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    if out is None:
        out = torch.empty(Wq.rows, Wq.cols, dtype=torch.bfloat16, device=Wq.codes.device)
    st = Wq.c_struct()
    _abi.check(_abi.lib().qlora_nf4_dequant(ctypes.byref(st), _ptr(out), _stream(out.device)),
               "qlora_nf4_dequant")
    return out


def workspace_bytes(M: int, N: int, K: int, r: int, dropout: bool = False) -> int:
    if dropout:
        return int(_abi.lib().qlora_linear_dropout_workspace_bytes(M, N, K, r))
    return int(_abi.lib().qlora_linear_workspace_bytes(M, N, K, r))


def make_workspace(M: int, N: int, K: int, r: int, device, dropout: bool = False,
                   checkpoint: bool = False) -> torch.Tensor:
    """Scratch of linear_fwd / linear_bwd; checkpoint: of linear_bwd with X an FP8Tensor
    (with or without dropout)."""
    if checkpoint:
        with torch.cuda.device(device):
            n = int(_abi.lib().qlora_linear_ckpt_workspace_bytes(M, N, K, r))
        return torch.empty(n, dtype=torch.uint8, device=device)
    return torch.empty(workspace_bytes(M, N, K, r, dropout), dtype=torch.uint8, device=device)


def pack_keep_mask(keep: torch.Tensor) -> torch.Tensor:
    """A boolean [M, K] keep mask as the library's bit-packed form: element m K + k in
    bit (m K + k) mod 8 of byte (m K + k) / 8 (uint8 [M K / 8], on keep's device).
    Marshalling only (torch bit operations)."""
    if keep.dim() != 2 or keep.shape[1] % 8:
        raise ValueError("keep must be [M, K] with K a multiple of 8")
    bits = keep.reshape(-1, 8).to(torch.uint8)
    w = torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], dtype=torch.uint8, device=keep.device)
    return (bits * w).sum(dim=1, dtype=torch.uint8).contiguous()


def _check_shapes(X: torch.Tensor, Wq: NF4Weight, A: torch.Tensor, B: torch.Tensor,
                  dY: Optional[torch.Tensor] = None) -> None:
    M, K = X.shape
    r = A.shape[1]
    if K != Wq.cols or A.shape[0] != Wq.cols or B.shape != (r, Wq.rows):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W [{Wq.rows}, {Wq.cols}], "
                         f"A {tuple(A.shape)}, B {tuple(B.shape)}")
    if dY is not None and dY.shape != (M, Wq.rows):
        raise ValueError(f"dY {tuple(dY.shape)} != ({M}, {Wq.rows})")


def linear_fwd(X: torch.Tensor, Wq: NF4Weight, A: torch.Tensor, B: torch.Tensor, s: float,
               workspace: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
               XA: Optional[torch.Tensor] = None, want_xa: bool = True,
               keep_bits: Optional[torch.Tensor] = None, dropout_p: float = 0.0):
    """Y = X deq(W)^T + s (X A) B  (bf16 [M, N]);  returns (Y, XA fp32 [M, r] or None).
    With keep_bits (pack_keep_mask of the [M, K] keep mask) the adapter input is
    X (.) keep / (1 - dropout_p)."""
    X = _bf16_2d(X, "X")
    A = _bf16_2d(A, "A")
    B = _bf16_2d(B, "B")
    _check_shapes(X, Wq, A, B)
    M = X.shape[0]
    r = A.shape[1]
    dev = X.device
    if Y is None:
        Y = torch.empty(M, Wq.rows, dtype=torch.bfloat16, device=dev)
    if XA is None and want_xa:
        XA = torch.empty(M, r, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = make_workspace(M, Wq.rows, Wq.cols, r, dev, dropout=keep_bits is not None)
    st = Wq.c_struct()
    if keep_bits is None:
        _abi.check(_abi.lib().qlora_linear_fwd(
            _ptr(X), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(s), _ptr(Y), _ptr(XA),
            _ptr(workspace), workspace.numel(), _stream(dev)), "qlora_linear_fwd")
    else:
        _abi.check(_abi.lib().qlora_linear_fwd_ex(
            _ptr(X), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(s), _ptr(keep_bits), float(dropout_p),
            _ptr(Y), _ptr(XA), _ptr(workspace), workspace.numel(), _stream(dev)), "qlora_linear_fwd_ex")
    return Y, XA


def linear_bwd(dY: torch.Tensor, X, XA: Optional[torch.Tensor], Wq: NF4Weight,
               A: torch.Tensor, B: torch.Tensor, s: float, need_dx: bool = True,
               workspace: Optional[torch.Tensor] = None, dX: Optional[torch.Tensor] = None,
               dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
               keep_bits: Optional[torch.Tensor] = None, dropout_p: float = 0.0,
               accumulate: bool = False):
    """Returns (dX bf16 [M, K] or None, dA fp32 [K, r], dB fp32 [r, N]).  keep_bits /
    dropout_p as in linear_fwd; accumulate adds into the given dA and dB.  X may be the
    8-bit checkpoint of the input (fp8_quantize(X)): dA = s deq(X)^T G."""
    if isinstance(X, FP8Tensor):
        return _linear_bwd_ckpt(dY, X, XA, Wq, A, B, s, need_dx, workspace, dX, dA, dB, keep_bits, dropout_p,
                                accumulate)
    if accumulate and (dA is None or dB is None):
        raise ValueError("accumulate needs the dA and dB to add into")
    dY = _bf16_2d(dY, "dY")
    X = _bf16_2d(X, "X")
    A = _bf16_2d(A, "A")
    B = _bf16_2d(B, "B")
    _check_shapes(X, Wq, A, B, dY)
    M = X.shape[0]
    r = A.shape[1]
    dev = X.device
    if dX is None and need_dx:
        dX = torch.empty(M, Wq.cols, dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty(Wq.cols, r, dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty(r, Wq.rows, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = make_workspace(M, Wq.rows, Wq.cols, r, dev, dropout=keep_bits is not None)
    st = Wq.c_struct()
    if keep_bits is None and not accumulate:
        _abi.check(_abi.lib().qlora_linear_bwd(
            _ptr(dY), _ptr(X), _ptr(XA), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(s),
            _ptr(dX), _ptr(dA), _ptr(dB), _ptr(workspace), workspace.numel(), _stream(dev)),
            "qlora_linear_bwd")
    else:
        _abi.check(_abi.lib().qlora_linear_bwd_ex(
            _ptr(dY), _ptr(X), _ptr(XA), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(s),
            _ptr(keep_bits), float(dropout_p), 1 if accumulate else 0,
            _ptr(dX), _ptr(dA), _ptr(dB), _ptr(workspace), workspace.numel(), _stream(dev)),
            "qlora_linear_bwd_ex")
    return dX, dA, dB


def nf4_merge(A: torch.Tensor, B: torch.Tensor, s: float, Wq: Optional[NF4Weight] = None,
              W16: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The adapter folded into a 16-bit weight: bf16(base + s (A B)^T) [N, K], base the
    bf16 original W16 or the dequantized Wq (pass exactly one)."""
    A = _bf16_2d(A, "A")
    B = _bf16_2d(B, "B")
    if (Wq is None) == (W16 is None):
        raise ValueError("pass exactly one of Wq and W16")
    if W16 is not None:
        W16 = _bf16_2d(W16, "W16")
        N, K = W16.shape
        dev = W16.device
    else:
        N, K = Wq.rows, Wq.cols
        dev = Wq.codes.device
    r = A.shape[1]
    if A.shape[0] != K or tuple(B.shape) != (r, N):
        raise ValueError(f"shape mismatch: W [{N}, {K}], A {tuple(A.shape)}, B {tuple(B.shape)}")
    if out is None:
        out = torch.empty(N, K, dtype=torch.bfloat16, device=dev)
    st = Wq.c_struct() if Wq is not None else None
    _abi.check(_abi.lib().qlora_nf4_merge(ctypes.byref(st) if st is not None else None, _ptr(W16), N, K,
                                          _ptr(A), _ptr(B), r, s, _ptr(out), _stream(dev)),
               "qlora_nf4_merge")
    return out


# ------------------------------------------------------------------ 8-bit floating point
# The current stream's handle by device index; the Stream object of the public call costs
# more than a small quantize does on the GPU.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name: str, dev: torch.device, *args) -> None:
    """The library function on dev's current stream, with dev current; None and pointers as
    integers in args."""
    fn = getattr(_abi.lib(), name)
    if torch.cuda.current_device() == dev.index:
        code = fn(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(dev.index))
    if code != _abi.QLORA_OK:
        raise _abi.QloraError(code, name)


def _dptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _out(t: Optional[torch.Tensor], shape: tuple, dtype: torch.dtype, dev, name: str) -> torch.Tensor:
    """The given output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} tensor on {dev}")
    return t


def _scratch(t: torch.Tensor, dev) -> Tuple[int, int]:
    """(pointer, bytes) of a workspace, checked."""
    if t.device != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _on(dev, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _saved_xa(XA: Optional[torch.Tensor], M: int, r: int) -> Optional[torch.Tensor]:
    if XA is None:
        return None
    if XA.dtype != torch.float32 or tuple(XA.shape) != (M, r):
        raise ValueError(f"XA must be float32 ({M}, {r})")
    return XA.contiguous()


def fp8_empty(rows: int, cols: int, device, fmt: str = "e4m3", block_rows: int = 1) -> FP8Tensor:
    if fmt not in _FP8_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(_FP8_FORMATS)}")
    return FP8Tensor(torch.empty(rows, cols, dtype=_FP8_FORMATS[fmt], device=device),
                     torch.empty(_fp8_scale_shape(rows, cols, block_rows), dtype=torch.uint8, device=device),
                     block_rows)


def _fp8_quantize(X: torch.Tensor, q: FP8Tensor) -> FP8Tensor:
    rows, cols = X.shape
    _call("qlora_fp8_quantize", X.device, X.data_ptr(), rows, cols, q.c_struct())
    return q


def fp8_quantize(X: torch.Tensor, fmt: str = "e4m3", out: Optional[FP8Tensor] = None) -> FP8Tensor:
    """A bf16 activation or gradient [M, K] in 8 bits, one power of two per 128 values of a
    row: the operand of fp8_linear_fwd and the checkpoint its backward reads.  With `out`
    given, its format is the one used."""
    X = _bf16_2d(X, "X")
    if out is None:
        out = fp8_empty(X.shape[0], X.shape[1], X.device, fmt)
    else:
        out.check("out", 1)
        if tuple(out.codes.shape) != tuple(X.shape) or out.device != X.device:
            raise ValueError(f"out {tuple(out.codes.shape)} on {out.device} does not match X {tuple(X.shape)}")
    return _fp8_quantize(X, out)


def fp8_quantize_weight(W: torch.Tensor, out: Optional[FP8Tensor] = None) -> FP8Tensor:
    """A frozen bf16 weight [N, K] in e4m3, one power of two per 128 x 128 block."""
    W = _bf16_2d(W, "W")
    if out is None:
        out = fp8_empty(W.shape[0], W.shape[1], W.device, "e4m3", 128)
    else:
        out.check("out", 128)
        if tuple(out.codes.shape) != tuple(W.shape) or out.device != W.device:
            raise ValueError(f"out {tuple(out.codes.shape)} on {out.device} does not match W {tuple(W.shape)}")
    return _fp8_quantize(W, out)


def fp8_dequant(X: FP8Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The bf16 values of an FP8Tensor."""
    rows, cols = X.check("X")
    out = _out(out, (rows, cols), torch.bfloat16, X.device, "out")
    _call("qlora_fp8_dequant", X.device, X.c_struct(), out.data_ptr())
    return out


def fp8_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(_abi.lib().qlora_fp8_workspace_bytes(M, N, K, r))


def fp8_make_workspace(M: int, N: int, K: int, r: int, device) -> torch.Tensor:
    """Scratch of fp8_linear_fwd / fp8_linear_bwd (r = 0: without an adapter)."""
    with torch.cuda.device(device):
        n = fp8_workspace_bytes(M, N, K, r)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _fp8_adapter(A, B, N: int, K: int):
    """(A, B, r) of an adapter, or (None, None, 0)."""
    if (A is None) != (B is None):
        raise ValueError("pass both A and B, or neither")
    if A is None:
        return None, None, 0
    A, B = _bf16_2d(A, "A"), _bf16_2d(B, "B")
    a_rows, r = A.shape
    if a_rows != K or B.shape != (r, N):
        raise ValueError(f"shape mismatch: W [{N}, {K}], A {tuple(A.shape)}, B {tuple(B.shape)}")
    return A, B, r


def fp8_linear_fwd(X: FP8Tensor, W: FP8Tensor, A: Optional[torch.Tensor] = None, B: Optional[torch.Tensor] = None,
                   s: float = 1.0, workspace: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                   XA: Optional[torch.Tensor] = None, want_xa: bool = True):
    """Y = deq(X) deq(W)^T + s (deq(X) A) B  (bf16 [M, N]) on an 8-bit frozen base; returns
    (Y, XA fp32 [M, r] or None).  Without A and B: the product alone."""
    M, K = X.check("X", 1)
    N, w_cols = W.check("W", 128)
    dev = X.codes.device
    A, B, r = _fp8_adapter(A, B, N, K)
    if w_cols != K:
        raise ValueError(f"shape mismatch: X [{M}, {K}], W [{N}, {w_cols}]")
    _on(dev, W=W.codes, A=A, B=B)
    Y = _out(Y, (M, N), torch.bfloat16, dev, "Y")
    if r and (XA is not None or want_xa):
        XA = _out(XA, (M, r), torch.float32, dev, "XA")
    elif XA is not None:
        raise ValueError("XA needs an adapter")
    if workspace is None:
        workspace = fp8_make_workspace(M, N, K, r, dev)
    _call("qlora_fp8_linear_fwd", dev, X.c_struct(), W.c_struct(), _dptr(A), _dptr(B), r, s,
          Y.data_ptr(), _dptr(XA), *_scratch(workspace, dev))
    return Y, XA


def fp8_linear_bwd(dY: torch.Tensor, X: Optional[FP8Tensor], XA: Optional[torch.Tensor], W: FP8Tensor,
                   A: Optional[torch.Tensor] = None, B: Optional[torch.Tensor] = None, s: float = 1.0,
                   need_dx: bool = True, grad_fmt: str = "e4m3", workspace: Optional[torch.Tensor] = None,
                   dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                   dB: Optional[torch.Tensor] = None, accumulate: bool = False):
    """Backward of fp8_linear_fwd: (dX bf16 [M, K] or None, dA fp32 [K, r], dB fp32 [r, N]).
    X is the forward's 8-bit input; the base product takes dY in blocks of 128 rounded to
    grad_fmt.  accumulate adds into the given dA and dB.  Without A and B (X and XA then
    unused): (dX, None, None)."""
    if grad_fmt not in _FP8_FORMATS:
        raise ValueError(f"grad_fmt must be one of {sorted(_FP8_FORMATS)}")
    dY = _bf16_2d(dY, "dY")
    N, K = W.check("W", 128)
    dev = dY.device
    M, dy_cols = dY.shape
    A, B, r = _fp8_adapter(A, B, N, K)
    if dy_cols != N:
        raise ValueError(f"dY {tuple(dY.shape)} does not match W [{N}, {K}]")
    if accumulate and (dA is None or dB is None):
        raise ValueError("accumulate needs the dA and dB to add into")
    if not r and (dA is not None or dB is not None or not need_dx):
        raise ValueError("dA and dB need an adapter; without one dX is the only result")
    xs = None
    if r:
        if X is None:
            raise ValueError("the adapter's gradients need X")
        if X.check("X", 1) != (M, K):
            raise ValueError(f"X [{X.rows}, {X.cols}] != ({M}, {K})")
        XA = _saved_xa(XA, M, r)
        xs = X.c_struct()
        _on(dev, X=X.codes, XA=XA, A=A, B=B)
        dA = _out(dA, (K, r), torch.float32, dev, "dA")
        dB = _out(dB, (r, N), torch.float32, dev, "dB")
    else:
        XA = None
    _on(dev, W=W.codes)
    dX = _out(dX, (M, K), torch.bfloat16, dev, "dX") if need_dx else None
    if workspace is None:
        workspace = fp8_make_workspace(M, N, K, r, dev)
    _call("qlora_fp8_linear_bwd", dev, dY.data_ptr(), M, xs, _dptr(XA), W.c_struct(), _dptr(A), _dptr(B), r, s,
          1 if grad_fmt == "e5m2" else 0, 1 if accumulate else 0, _dptr(dX), _dptr(dA), _dptr(dB),
          *_scratch(workspace, dev))
    return dX, dA, dB


def _linear_bwd_ckpt(dY, X: FP8Tensor, XA, Wq: NF4Weight, A, B, s, need_dx, workspace, dX, dA, dB, keep_bits,
                     dropout_p, accumulate):
    """linear_bwd with the saved input in 8 bits."""
    dY = _bf16_2d(dY, "dY")
    M, x_cols = X.check("X", 1)
    N, K = Wq.rows, Wq.cols
    A, B, r = _fp8_adapter(A, B, N, K)
    if not r:
        raise ValueError("linear_bwd needs A and B")
    dev = dY.device
    if x_cols != K or dY.shape != (M, N):
        raise ValueError(f"shape mismatch: dY {tuple(dY.shape)}, X [{M}, {x_cols}], W [{N}, {K}]")
    if accumulate and (dA is None or dB is None):
        raise ValueError("accumulate needs the dA and dB to add into")
    if keep_bits is not None and (keep_bits.dtype != torch.uint8 or not keep_bits.is_contiguous()
                                  or keep_bits.numel() * 8 < M * K):
        raise ValueError("keep_bits must be the packed mask (uint8) of the M x K input")
    XA = _saved_xa(XA, M, r)
    _on(dev, X=X.codes, XA=XA, W=Wq.codes, A=A, B=B, keep_bits=keep_bits)
    dX = _out(dX, (M, K), torch.bfloat16, dev, "dX") if need_dx else None
    dA = _out(dA, (K, r), torch.float32, dev, "dA")
    dB = _out(dB, (r, N), torch.float32, dev, "dB")
    if workspace is None:
        workspace = make_workspace(M, N, K, r, dev, checkpoint=True)
    _call("qlora_linear_bwd_ckpt", dev, dY.data_ptr(), X.c_struct(), _dptr(XA),
          ctypes.byref(Wq.c_struct()), A.data_ptr(), B.data_ptr(), r, s, _dptr(keep_bits), dropout_p,
          1 if accumulate else 0, _dptr(dX), dA.data_ptr(), dB.data_ptr(), *_scratch(workspace, dev))
    return dX, dA, dB


def device_status(sync_stream: bool = True) -> Tuple[int, int]:
    """(status code, flags) of the current device; reads and clears the word."""
    flags = ctypes.c_uint32(0)
    code = _abi.lib().qlora_get_device_status(_stream(), ctypes.byref(flags))
    return code, flags.value


def selftest_wait_timeout(timeout_us: int) -> int:
    return _abi.lib().qlora_selftest_wait_timeout(timeout_us, _stream())


def set_wait_limit_us(limit_us: int) -> int:
    return int(_abi.lib().qlora_set_wait_limit_us(limit_us))


def gemm_units() -> tuple:
    """(single CTAs, CTA pairs) the fused GEMM runs on this device."""
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    _abi.check(_abi.lib().qlora_gemm_units(ctypes.byref(a), ctypes.byref(b)), "qlora_gemm_units")
    return a.value, b.value


def set_gemm_pairing(enable: bool) -> bool:
    """Two-CTA (256-row) GEMM tiles where the output width allows; returns the previous setting."""
    return bool(_abi.lib().qlora_set_gemm_pairing(1 if enable else 0))


def profile_enable(on: bool = True) -> None:
    """Record CUDA events around every launch of the library's kernels."""
    _abi.check(_abi.lib().qlora_profile_enable(1 if on else 0), "qlora_profile_enable")


def profile_read():
    """[(kernel kind name, milliseconds)] of the launches recorded since enabling
    (oldest first, at most the ring capacity) and the total launch count."""
    cap = _abi.PROFILE_CAP
    kinds = (ctypes.c_int * cap)()
    ms = (ctypes.c_float * cap)()
    n = _abi.lib().qlora_profile_read(cap, kinds, ms)
    if n < 0:
        raise RuntimeError("qlora_profile_read failed")
    k = min(n, cap)
    return [(_abi.KERNEL_KINDS[kinds[i]], float(ms[i])) for i in range(k)], n
