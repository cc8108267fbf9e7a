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


# ------------------------------------------------------------------ accumulation
@pytest.mark.parametrize("M,N,K,r", [(70, 256, 384, 16), (300, 384, 512, 72), (260, 512, 384, 128)])
@pytest.mark.parametrize("saved", [True, False])
def test_accumulation_on_the_8_bit_layer(q, M, N, K, r, saved):
    """Three micro-batches added into the same dA and dB, dX wanted each time: the gradients of each alone
    added in fp32 in their order, and dX of each alone."""
    import torch
    ps = [Problem(M, N, K, r, seed=i) for i in range(3)]
    Wq, A, B = q.fp8_quantize_weight(dev(ps[0].W)), dev(ps[0].A), dev(ps[0].B)
    ws = q.fp8_make_workspace(M, N, K, r, "cuda")
    dA, dB = torch.full((K, r), 0.5, device="cuda"), torch.full((r, N), -0.25, device="cuda")
    wantA, wantB = dA.clone(), dB.clone()
    for p in ps:
        Xq, dY = q.fp8_quantize(dev(p.X)), dev(p.dY)
        XA = q.fp8_linear_fwd(Xq, Wq, A, B, p.s, workspace=ws)[1] if saved else None
        dX1, a, b = q.fp8_linear_bwd(dY, Xq, XA, Wq, A, B, p.s, workspace=ws)
        dX2, _, _ = q.fp8_linear_bwd(dY, Xq, XA, Wq, A, B, p.s, workspace=ws, dA=dA, dB=dB, accumulate=True)
        wantA += a
        wantB += b
        assert same([dX1], [dX2])
    torch.cuda.synchronize()
    assert q.device_status() == (0, 0)
    assert torch.equal(dA, wantA) and torch.equal(dB, wantB)


# ------------------------------------------------------------------ the NF4 layer from an 8-bit checkpoint
def packed(keep):
    import torch
    return torch.from_numpy(np.packbits(keep.astype(np.uint8).ravel(), bitorder="little")).cuda()


@pytest.mark.parametrize("M,N,K,r,pdrop", [(5, 256, 384, 16, 0.0), (300, 384, 256, 24, 0.0), (270, 512, 640, 72, 0.1)])
@pytest.mark.parametrize("saved", [True, False])
def test_checkpoint_on_single_level_constants(q, M, N, K, r, pdrop, saved):
    import helpers as H
    import torch
    from fp8_problems import host, product_check
    from oracle import linear as olin
    p = Problem(M, N, K, r, span=2)
    A, B, dY, X = dev(p.A), dev(p.B), dev(p.dY), dev(p.X)
    Wq = q.nf4_quantize(dev(p.W), single_level=True)
    assert Wq.single_level
    keep = np.random.default_rng(M).random((M, K)) >= pdrop
    kw = dict(keep_bits=packed(keep), dropout_p=pdrop) if pdrop else {}
    XA = q.linear_fwd(X, Wq, A, B, p.s, **kw)[1]
    dX, dA, dB = q.linear_bwd(dY, q.fp8_quantize(X), XA if saved else None, Wq, A, B, p.s, **kw)
    torch.cuda.synchronize()
    assert q.device_status() == (0, 0)
    Wd, G, kf = host(q.nf4_dequant(Wq)), p.dY @ p.B.T, keep / (1.0 - pdrop)
    term = p.s * (G @ p.A.T) * kf
    mag = np.abs(p.dY) @ np.abs(Wd) + p.s * (np.abs(G) @ np.abs(p.A).T) * kf
    assert product_check(host(dX), p.dY @ Wd + term, mag, 2 * N) <= 1.0
    Xin = p.Xd * kf
    XAr = host(XA) if saved else Xin @ p.A
    g = olin.backward(p.dY, Xin, np.zeros((N, K)), p.A, p.B, p.s, XA=XAr)
    mags = H.lora_magnitudes(Xin, p.A, p.B, p.dY, p.s, XA=XAr)
    for name, got in (("dA", dA), ("dB", dB)):
        assert H.mag_check(host(got), g[name], mags[name]) <= 1.0, name


@pytest.mark.parametrize("M,N,K,r,pdrop", [(3, 512, 384, 16, 0.0), (300, 512, 768, 24, 0.1), (700, 9728, 256, 72, 0.0)])
def test_checkpoint_in_graphs_and_on_streams(q, M, N, K, r, pdrop):
    """quantize, forward and the backward from the checkpoint: three streams at once, then two graphs
    replayed in turn on new inputs; every result is the one of a call alone."""
    import torch
    ps = [Problem(M, N, K, r, seed=i) for i in range(2)]
    Wq, A, B, s = q.nf4_quantize(dev(ps[0].W)), dev(ps[0].A), dev(ps[0].B), ps[0].s
    keep = np.random.default_rng(M).random((M, K)) >= pdrop
    kw = dict(keep_bits=packed(keep), dropout_p=pdrop) if pdrop else {}

    def spaces():
        return (q.make_workspace(M, N, K, r, "cuda", dropout=bool(pdrop)), q.make_workspace(M, N, K, r, "cuda", checkpoint=True))

    def step(X, dY, ws):
        Xq = q.fp8_quantize(X)
        Y, XA = q.linear_fwd(X, Wq, A, B, s, workspace=ws[0], **kw)
        return (Y, XA, *q.linear_bwd(dY, Xq, XA, Wq, A, B, s, workspace=ws[1], **kw),
                *q.linear_bwd(dY, Xq, None, Wq, A, B, s, workspace=ws[1], **kw))

    ins = [(dev(p.X), dev(p.dY)) for p in ps]
    want = [step(*i, spaces()) for i in ins]
    torch.cuda.synchronize()
    streams, ws, got = [torch.cuda.Stream() for _ in range(3)], [spaces() for _ in range(3)], []
    for rep in range(6):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(((rep + k) % 2, step(*ins[(rep + k) % 2], ws[k])))
    torch.cuda.synchronize()
    assert all(same(g, want[i]) for i, g in got)
    bufs = [tuple(torch.zeros_like(t) for t in ins[0]) for _ in range(2)]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*bufs[i], ws[i]))
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for gi, which in enumerate(order):
            for b, t in zip(bufs[gi], ins[which]):
                b.copy_(t)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(same(outs[gi], want[which]) for gi, which in enumerate(order))
    assert q.device_status() == (0, 0)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_checkpoint_with_a_non_finite_gradient(q, bad):
    """One element of dY: its token's dX and its output's dB are not finite, all other tokens' dX and
    outputs' dB keep their bits."""
    import torch
    M, N, K, r = 300, 256, 384, 16
    p = Problem(M, N, K, r)
    Xq, W4, A, B, dY = q.fp8_quantize(dev(p.X)), q.nf4_quantize(dev(p.W)), dev(p.A), dev(p.B), dev(p.dY)
    XA = q.linear_fwd(dev(p.X), W4, A, B, p.s)[1]
    ref = [t.clone() for t in q.linear_bwd(dY, Xq, XA, W4, A, B, p.s)]
    dY[133, 200] = bad
    dX, dA, dB = q.linear_bwd(dY, Xq, XA, W4, A, B, p.s)
    torch.cuda.synchronize()
    tok = torch.arange(M, device="cuda") != 133
    col = torch.arange(N, device="cuda") != 200
    assert not torch.isfinite(dX[133].float()).any() and torch.equal(dX[tok], ref[0][tok])
    assert not torch.isfinite(dB[:, 200]).any() and torch.equal(dB[:, col], ref[2][:, col])
    assert not torch.isfinite(dA).any()
    q.device_status()


# ------------------------------------------------------------------ one call's result as the next one's input
@pytest.mark.parametrize("M", [1, 8, 13, 100, 300])
@pytest.mark.parametrize("r", [0, 16, 72])
def test_calls_that_read_what_the_call_before_wrote(q, M, r):
    """Layer after layer, forward and backward, launched back to back without a kernel of another kind
    between them: each reads what the launch before has just written.  Twenty rounds over changing
    inputs, with the same bits as one call at a time with the GPU waited for."""
    import torch
    N = K = 512
    ps = [Problem(M, N, K, r, seed=i, span=1) for i in range(3)]
    Wq = [q.fp8_quantize_weight(dev(p.W)) for p in ps]
    ad = [(dev(p.A), dev(p.B), p.s) if r else () for p in ps]
    xs, dys = [dev(p.X) for p in ps], [dev(p.dY) for p in ps]
    ws = q.fp8_make_workspace(M, N, K, r, "cuda")

    def run(i, wait):
        h, saved, out = xs[i], [], []

        def after(*t):
            out.extend(t)
            if wait:
                torch.cuda.synchronize()

        for W, a in zip(Wq, ad):
            Xq = q.fp8_quantize(h)
            after(Xq.codes, Xq.scales)
            h, XA = q.fp8_linear_fwd(Xq, W, *a, workspace=ws)
            after(h, XA)
            saved.append((Xq, XA))
        g = dys[i]
        for W, a, (Xq, XA) in reversed(list(zip(Wq, ad, saved))):
            g, dA, dB = q.fp8_linear_bwd(g, Xq if r else None, XA, W, *a, grad_fmt="e5m2", workspace=ws)
            after(g, dA, dB)
        return out

    want = [run(i, True) for i in range(3)]
    got = [(i % 3, run(i % 3, False)) for i in range(20)]
    torch.cuda.synchronize()
    assert q.device_status() == (0, 0)
    assert all(same(g, want[i]) for i, g in got)


# ------------------------------------------------------------------ which form a forward takes
@pytest.mark.parametrize("M,r,few", [(1, 0, True), (8, 48, True), (8, 64, False), (6, 64, True), (8, 72, True), (8, 128, True),
                                     (3, 128, True), (9, 0, False), (9, 128, False)])
def test_few_token_form_by_tokens_and_rank(q, M, r, few):
    """Up to 8 tokens: the few-token kernel while M r <= 384, and for every rank past 64, where the GEMM's
    form needs two passes for XA."""
    import torch
    p = Problem(M, 256, 384, r)
    Xq, Wq = q.fp8_quantize(dev(p.X)), q.fp8_quantize_weight(dev(p.W))
    ad = (dev(p.A), dev(p.B), p.s) if r else ()
    q.profile_enable(True)
    try:
        q.fp8_linear_fwd(Xq, Wq, *ad)
        torch.cuda.synchronize()
        kinds = [k for k, _ in q.profile_read()[0]]
    finally:
        q.profile_enable(False)
    assert ("fp8_skinny" in kinds) == few and ("fp8_gemm_fwd" in kinds) == (not few)
