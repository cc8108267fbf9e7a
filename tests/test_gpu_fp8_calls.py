"""Calls of the 8-bit operators, and of the NF4 layer from an 8-bit checkpoint, that the documentation
allows beyond the ordinary ones."""
import numpy as np
import pytest

from fp8_problems import Problem, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_19_b200 as q
    from bit_nf4_quantized_19_b200 import build
    build.build()
    return q


def bits(t):
    import torch
    return t.contiguous().view(torch.uint8)


def same(a, b):
    import torch
    return all((x is None and y is None) or torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


# ------------------------------------------------------------------ workspaces
@pytest.mark.parametrize("M,N,K,r", [(3, 256, 384, 16), (60, 384, 2176, 24), (300, 512, 384, 72), (200, 4096, 256, 16)])
def test_workspace_at_any_16_byte_start(q, M, N, K, r):
    """A workspace of exactly the queried size at every 16-byte start, between guards: the same bits as
    from one of its own, and the guards stay."""
    import torch
    p = Problem(M, N, K, r)
    X, A, B, dY = dev(p.X), dev(p.A), dev(p.B), dev(p.dY)
    Xq, Wq, W4 = q.fp8_quantize(X), q.fp8_quantize_weight(dev(p.W)), q.nf4_quantize(dev(p.W))
    keep = torch.arange(M * K // 8, device="cuda", dtype=torch.int64).mul(37).to(torch.uint8)
    drop = dict(keep_bits=keep, dropout_p=0.1)
    sizes = dict(fp8=q.fp8_workspace_bytes(M, N, K, r), ckpt=q.make_workspace(M, N, K, r, "cuda", checkpoint=True).numel(),
                 nf4=q.workspace_bytes(M, N, K, r), drop=q.workspace_bytes(M, N, K, r, True))

    def calls(ws):
        Y, XA = q.fp8_linear_fwd(Xq, Wq, A, B, p.s, workspace=ws("fp8"))
        out = [Y, XA, *q.fp8_linear_bwd(dY, Xq, XA, Wq, A, B, p.s, workspace=ws("fp8"))]
        out += q.fp8_linear_bwd(dY, Xq, None, Wq, A, B, p.s, grad_fmt="e5m2", workspace=ws("fp8"))
        Y, XA = q.linear_fwd(X, W4, A, B, p.s, workspace=ws("nf4"))
        out += [Y, XA, *q.linear_bwd(dY, X, XA, W4, A, B, p.s, workspace=ws("nf4"))]
        out += q.linear_bwd(dY, Xq, XA, W4, A, B, p.s, workspace=ws("ckpt"))
        out += q.linear_bwd(dY, Xq, None, W4, A, B, p.s, workspace=ws("ckpt"), **drop)
        out += q.linear_fwd(X, W4, A, B, p.s, workspace=ws("drop"), **drop)
        return out

    want = calls(lambda kind: torch.empty(sizes[kind], dtype=torch.uint8, device="cuda"))
    buf = torch.full((max(sizes.values()) + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    for start in range(16, 272, 16):
        buf.fill_(0xA5)
        used = []

        def view(kind):
            # each kind's guards are checked before the next takes the buffer
            while used:
                k = used.pop()
                assert (buf[:start] == 0xA5).all() and (buf[start + sizes[k]:] == 0xA5).all(), (start, k)
            buf[start + sizes[kind]:].fill_(0xA5)
            used.append(kind)
            return buf[start:start + sizes[kind]]

        got = calls(view)
        torch.cuda.synchronize()
        assert same(want, got), start
    assert q.device_status() == (0, 0)


# ------------------------------------------------------------------ factors far from one on both operands
FORMS = [1, 8, 12, 100, 300]      # tokens: the few-token kernel, the weight on the MMA's rows, whole tiles


@pytest.mark.parametrize("M", FORMS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_large_factors_on_both_operands(q, M, fmt):
    """Two blocks meet whose factors' product passes 2^128.  Rows of W without a value there, and rows
    whose product is still a bf16 value, are what the formula gives; only the row whose product
    is past bf16 is infinite.  Every product and sum is exact but for the rounding to bf16."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 256, 512
    X = rng.integers(-4, 5, (M, K)).astype(np.float64)
    X[:, :128] = 0.0
    X[:, 0], X[:, 1] = 2.0 ** 106, 2.0 ** 90      # the first sets the block's factor, 2^98 or 2^91
    W = rng.integers(-4, 5, (N, K)).astype(np.float64)
    W[:, :128] = 0.0                              # rows 128 ..: a block of zeros, factor 2^-127
    W[5, 0] = 2.0 ** 48                           # sets its block's factor, 2^40
    W[7:128, 1] = 2.0 ** 32
    Xq, Wq = q.fp8_quantize(dev(X), fmt=fmt), q.fp8_quantize_weight(dev(W))
    assert int(Xq.scales[0, 0]) + int(Wq.scales[0, 0]) - 254 == (138 if fmt == "e4m3" else 131)
    with np.errstate(over="ignore"):
        want = torch.from_numpy((X @ W.T).astype(np.float32)).to(torch.bfloat16)
    Y, _ = q.fp8_linear_fwd(Xq, Wq)
    torch.cuda.synchronize()
    assert q.device_status() == (0, 0)
    assert torch.isinf(want[:, 5]).all() and torch.isfinite(want).sum() == M * (N - 1)
    assert torch.equal(Y.cpu(), want)


@pytest.mark.parametrize("M", FORMS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_small_factors_on_both_operands(q, M, fmt):
    """Two blocks meet whose factors' product is below 2^-149, fp32's smallest, while the sum of their
    codes' products brings it back: 1024 products of (FMAX 2^-a) (448 2^-75) are 1.5 2^-123 (e4m3) or
    1.5 2^-126, normal bf16 values; in the other rows they come with a sign."""
    import torch
    N, K = 256, 1024
    top, a = (448.0, 75) if fmt == "e4m3" else (57344.0, 85)
    sign = np.where(np.arange(N) % 3 == 0, -1.0, 1.0)
    X, W = np.full((M, K), top * 2.0 ** -a), np.full((N, K), 448.0 * 2.0 ** -75) * sign[:, None]
    Xq, Wq = q.fp8_quantize(dev(X), fmt=fmt), q.fp8_quantize_weight(dev(W))
    assert int(Xq.scales[0, 0]) + int(Wq.scales[0, 0]) - 254 == -75 - a
    want = torch.from_numpy(X @ W.T).to(torch.bfloat16)
    assert torch.equal(want.double(), torch.from_numpy(X @ W.T))
    Y, _ = q.fp8_linear_fwd(Xq, Wq)
    torch.cuda.synchronize()
    assert q.device_status() == (0, 0)
    assert torch.equal(Y.cpu(), want)
