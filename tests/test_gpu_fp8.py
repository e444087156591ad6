"""moe_fp8_quantize, moe_fp8_quantize_weights, moe_fp8_gemm and moe_fp8_linear
(forward and backward) against plain implementations.

Bars.  Codes and scales: bit-exact (each is a correctly rounded operation).
Products.  The matrix cores align a chunk's 128 products to the largest of them
and drop what lies far below it: where products span many binades a chunk's sum
is off by up to 3.8e-4 of its largest product (16384 outputs of uniformly drawn
codes; 2.0e-4 with codes of normal numbers), so 2^-10 of the product of the two
rows' largest magnitudes is allowed per chunk.  Products within a few binades
are summed exactly: with codes of +-{0.5, 1, 1.5, 2} the fp32 operations are
all that is left, one for the scales' product and one fma per chunk,
(chunks + 2) 2^-24 of the sum of magnitudes.  A bf16 result adds 2^-8 of its value (half
an ulp is 2^-9, and as much for the error that moves it)."""
import math

import numpy as np
import pytest
import torch

from fp4_weight_grouped_amd import v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _float32():
    """Other modules set another default type when they are collected."""
    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(old)


def up(n, m):
    return (n + m - 1) // m * m


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def quant_ref(x, rows, cols):
    """Codes and scales of x with a scale for each rows x cols tile, fp32 operations on the CPU."""
    R, C = x.shape
    v = np.zeros((up(R, rows), up(C, cols)), np.float32)
    v[:R, :C] = x.float().cpu().numpy()
    t = v.reshape(v.shape[0] // rows, rows, v.shape[1] // cols, cols)
    s = (np.abs(t).max(axis=(1, 3)) / np.float32(448)).astype(np.float32)
    s[s == 0] = 1
    q = np.clip(t / s[:, None, :, None], -448, 448).reshape(v.shape)[:R, :C]
    code = torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).view(torch.uint8)
    return code, torch.from_numpy(s)


def source(seed, R, C, type, pad=0, at=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=g) * torch.exp(torch.randn(R, 1, generator=g) * 2)
    if R > 3 and C > 3:
        x[1] = 0
        x[2, : C // 2] = 0
        x[3] *= 1e-42                   # fp32 subnormals
    wide = torch.zeros(R, C + pad + at, dtype=type, device=DEV)
    wide[:, at:at + C] = x.to(type).to(DEV)
    return wide[:, at:at + C]


SHAPES = [(1, 1), (1, 128), (3, 17), (16, 256), (127, 129), (128, 128), (130, 1000), (257, 384), (1, 4096), (1000, 31)]


@pytest.mark.parametrize("type", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize(shape, type):
    R, C = shape
    for pad, at in ((0, 0), (5, 0), (16, 8), (3, 1)):
        x = source(R + C, R, C, type, pad, at)
        for rows, cols in ((True, False), (False, True), (True, True)):
            q, s, qt, st = v4moe.fp8_quantize(x, rows, cols)
            if rows:
                rq, rs = quant_ref(x, 1, 128)
                assert torch.equal(q[:, :C].cpu(), rq) and torch.equal(s.cpu(), rs.t())
                assert not q[:, C:].any()
            if cols:
                rq, rs = quant_ref(x.t(), 1, 128)
                assert torch.equal(qt[:, :R].cpu(), rq) and torch.equal(st.cpu(), rs.t())
                assert not qt[:, R:].any()
    m = v4moe.fp8_weights(x)
    rq, rs = quant_ref(x, 128, 128)
    assert torch.equal(m.q[:, :C].cpu(), rq) and torch.equal(m.blk.cpu(), rs) and not m.q[:, C:].any()
    assert torch.equal(m.qt[:, :R].cpu(), rq.t()) and not m.qt[:, R:].any()


def test_quantize_not_finite():
    for bad in (math.inf, -math.inf, math.nan):
        x = source(5, 300, 300, torch.float32)
        x[140, 200] = bad
        q, s, qt, st = v4moe.fp8_quantize(x, True, True)
        assert s.isnan().sum() == 1 and bool(s[1, 140].isnan()) and not q[140, 128:256].any()
        assert st.isnan().sum() == 1 and bool(st[1, 200].isnan()) and not qt[200, 128:256].any()
        w = v4moe.fp8_weights(torch.ones(64, 300, device=DEV))
        y = v4moe.fp8_linear(x, w)
        assert bool(y[140].isnan().all()) and y.isnan().sum() == 64
        m = v4moe.fp8_weights(x)
        assert m.blk.isnan().sum() == 1 and bool(m.blk[1, 1].isnan())


def gemm_ref(a, sa, b, sb, wide):
    """64-bit result and the error allowed for fp32 chunk sums; sa [M][chunks], sb [N][chunks].  wide: codes of
    any magnitude (otherwise +-{0.5, 1, 1.5, 2} and zero)."""
    K = a.shape[1]
    ka = torch.arange(K, device=a.device) // 128
    A, B = values(a) * sa.double()[:, ka], values(b) * sb.double()[:, ka]
    mag = A.abs() @ B.abs().t()
    tol = mag * (up(K, 128) // 128 + 2) * 2.0 ** -24
    if wide:
        pad = up(K, 128) - K
        big = lambda v: torch.nn.functional.pad(v.abs(), (0, pad)).view(v.shape[0], -1, 128).amax(-1)  # noqa: E731
        tol = tol + big(A) @ big(B).t() * 2.0 ** -10
    return A @ B.t(), tol


def bar(ref, tol, type):
    return tol + (ref.abs() * 2.0 ** -8 if type == torch.bfloat16 else 0) + 1e-30


def operand(seed, R, C, pad=0, wide=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(0, 256, (R, C + pad), generator=g, device=DEV, dtype=torch.int32)
    if wide:
        q[(q & 127) == 127] = 5          # no NaN codes inside
    else:
        q = (q & 128) | (0x30 + 4 * (q & 3))
    q = q.to(torch.uint8)
    if pad:
        q[:, C:] = 0x7F                   # NaN codes beside
    s = torch.rand(R, max(1, up(C, 128) // 128), generator=g, device=DEV) + 0.1
    return q[:, :C], s


GEMMS = [(1, 1, 16), (1, 64, 128), (2, 17, 144), (5, 300, 1008), (16, 128, 2048), (17, 129, 256), (33, 48, 4096),
         (64, 256, 512), (65, 1000, 384), (100, 31, 112), (128, 512, 640), (129, 257, 272), (200, 384, 128),
         (300, 640, 1040), (513, 514, 528), (700, 1030, 256), (1100, 900, 384), (2050, 1300, 160), (1, 2000, 2064),
         (20, 1500, 272), (70, 2200, 1200), (300, 3000, 256), (1000, 3100, 144), (4100, 4000, 400),
         (4001, 3900, 272), (3990, 4090, 400)]


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("shape", GEMMS, ids=str)
def test_gemm(shape, wide, rows):
    M, N, K = shape
    for pad, type in ((0, torch.bfloat16), (48, torch.float32)):
        a, sa = operand(M, M, K, pad, wide)
        b, sb = operand(N + 7, N, K, pad, wide)
        if not rows:
            blk = sb[::128].contiguous()
            sb = blk.repeat_interleave(128, 0)[:N]
        sb_arg = sb.t().contiguous() if rows else blk
        ref, tol = gemm_ref(a, sa, b, sb, wide)
        for ldc in (N, N + 3):
            buf = torch.full((M, ldc), 3.0, dtype=type, device=DEV)
            out = v4moe.fp8_gemm(a, sa.t().contiguous(), b, sb_arg, rows, out=buf[:, :N])
            assert bool(((out.double() - ref).abs() <= bar(ref, tol, type)).all())
            assert bool((buf[:, N:] == 3).all())
        if not rows:                     # block scales read with other strides
            out2 = v4moe.fp8_gemm(a, sa.t().contiguous(), b, blk.t().contiguous().t(), False, out=torch.empty_like(out))
            assert torch.equal(out2, out)
        if type == torch.float32:
            acc = out.clone()
            v4moe.fp8_gemm(a, sa.t().contiguous(), b, sb_arg, rows, out=acc, accumulate=True)
            assert torch.equal(acc, out + out)


@pytest.mark.parametrize("shape", [(2050, 1300, 1056), (1100, 257, 4096), (4352, 4096, 656), (4001, 3800, 656)], ids=str)
@pytest.mark.parametrize("rows", [False, True])
def test_row_does_not_depend_on_the_batch(shape, rows):
    M, N, K = shape
    a, sa = operand(1, M, K, 0, True)
    b, sb = operand(2, N, K, 0, True)
    sb = sb.t().contiguous() if rows else sb[::128].contiguous()
    full = v4moe.fp8_gemm(a, sa.t().contiguous(), b, sb, rows, out=torch.empty(M, N, device=DEV))
    for lo, n in ((0, 1), (7, 5), (100, 16), (90, 33), (11, 64), (500, 100), (0, 200), (64, 400), (30, 700), (1000, 3000)):
        if lo + n > M:
            continue
        part = v4moe.fp8_gemm(a[lo:lo + n], sa[lo:lo + n].t().contiguous(), b, sb, rows, out=torch.empty(n, N, device=DEV))
        assert torch.equal(part, full[lo:lo + n]), (lo, n)


def test_gemm_edges():
    a, sa = operand(1, 40, 0)
    b, sb = operand(2, 30, 0)
    c = torch.ones(40, 30, device=DEV)
    g = v4moe.GemmC(40, 30, 0, 0, 0, 1, 0, 0, 30, 1, 1)
    P = v4moe._p
    assert v4moe.lib().moe_fp8_gemm(v4moe.ctypes.byref(g), None, None, None, None, P(c), v4moe._stream()) == 0
    assert bool((c == 1).all())          # accumulate: unchanged
    g.accumulate = 0
    assert v4moe.lib().moe_fp8_gemm(v4moe.ctypes.byref(g), None, None, None, None, P(c), v4moe._stream()) == 0
    assert not c.any()
    w = v4moe.fp8_weights(torch.randn(32, 48, device=DEV))
    x = torch.zeros(0, 48, device=DEV)
    assert v4moe.fp8_linear(x, w).shape == (0, 32)
    dx, dw = v4moe.fp8_linear_backward(x, torch.zeros(0, 32, device=DEV), w)
    assert dx.shape == (0, 48) and not dw.any()


@pytest.mark.parametrize("shape", [(1, 128, 256), (9, 77, 130), (130, 200, 1001), (515, 384, 640)], ids=str)
@pytest.mark.parametrize("type", [torch.float32, torch.bfloat16])
def test_linear(shape, type):
    M, N, K = shape
    x, w0 = source(1, M, K, type, 8, 0), source(2, N, K, torch.float32)
    dy = source(3, M, N, type, 16, 8)
    w = v4moe.fp8_weights(w0)
    blk = lambda t: t.repeat_interleave(128, 0)  # noqa: E731
    y = v4moe.fp8_linear(x, w)
    q, s = quant_ref(x, 1, 128)
    ref, tol = gemm_ref(q.to(DEV), s.to(DEV), w.q[:, :K], blk(w.blk)[:N], True)
    assert bool(((y.double() - ref).abs() <= bar(ref, tol, torch.bfloat16)).all())
    dw32 = torch.ones(N, K, device=DEV)
    dx, dw = v4moe.fp8_linear_backward(x, dy, w)
    v4moe.fp8_linear_backward(x, dy, w, dw=dw32, accumulate=True)
    q, s = quant_ref(dy, 1, 128)
    ref, tol = gemm_ref(q.to(DEV), s.to(DEV), w.qt[:, :N], blk(w.blk.t())[:K], True)
    assert bool(((dx.double() - ref).abs() <= bar(ref, tol, torch.bfloat16)).all())
    (qy, sy), (qx, sx) = quant_ref(dy.t(), 1, 128), quant_ref(x.t(), 1, 128)
    ref, tol = gemm_ref(qy.to(DEV), sy.to(DEV), qx.to(DEV), sx.to(DEV), True)
    assert bool(((dw.double() - ref).abs() <= bar(ref, tol, torch.bfloat16)).all())
    assert bool(((dw32.double() - 1 - ref).abs() <= bar(ref, tol, torch.float32) + 2.0 ** -23 * (1 + ref.abs())).all())


@pytest.mark.parametrize("shape", [(1, 128, 256), (40, 300, 520), (300, 1000, 900), (1237, 999, 1001), (700, 2100, 130),
                                   (2100, 1500, 3000), (130, 4100, 4000)], ids=str)
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_is_its_products(shape, accumulate):
    """Both gradients in one launch or two, alone or together: the bits of the products of the quantised operands."""
    M, N, K = shape
    x, dy = source(5, M, K, torch.bfloat16), source(6, M, N, torch.bfloat16)
    w = v4moe.fp8_weights(source(7, N, K, torch.float32))
    q, s, qt, st = v4moe.fp8_quantize(dy, True, True)
    _, _, xt, xts = v4moe.fp8_quantize(x, False, True)
    old = torch.randn(N, K, device=DEV)
    rdx = v4moe.fp8_gemm(q, s, w.qt, w.blk.t(), False, out=torch.empty(M, K, dtype=torch.bfloat16, device=DEV))
    rdw = v4moe.fp8_gemm(qt, st, xt, xts, True, out=torch.empty(N, K, device=DEV))
    dx, dw = v4moe.fp8_linear_backward(x, dy, w, dw=old.clone(), accumulate=accumulate)
    assert torch.equal(dx, rdx) and torch.equal(dw, rdw + old if accumulate else rdw)


@pytest.mark.parametrize("shape", [(5, 70, 200), (300, 520, 390), (1030, 1500, 2100)], ids=str)
@pytest.mark.parametrize("types", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16),
                                   (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)], ids=str)
def test_backward_of_one_operand(shape, types):
    """dx or dW alone, x and dy of either type: the bits of both together."""
    M, N, K = shape
    x, dy = source(5, M, K, types[0], 3, 1), source(6, M, N, types[1], 8)
    w = v4moe.fp8_weights(source(7, N, K, torch.float32))
    dx, dw = v4moe.fp8_linear_backward(x, dy, w)
    n = v4moe.moe_fp8_linear_workspace_bytes(M, N, K, 1)
    ws, P, c = torch.empty(n, dtype=torch.uint8, device=DEV), v4moe._p, w.c()
    code = {torch.float32: v4moe.TYPE_F32, torch.bfloat16: v4moe.TYPE_BF16}
    args = (P(x), code[types[0]], x.stride(0), P(dy), code[types[1]], dy.stride(0), v4moe.ctypes.byref(c))
    for one in (dx, dw):
        got = torch.empty_like(one)
        to = (P(got), v4moe.TYPE_BF16, K, None, v4moe.TYPE_BF16, K) if one is dx else (None, v4moe.TYPE_BF16, K, P(got), v4moe.TYPE_BF16, K)
        assert v4moe.lib().moe_fp8_linear_backward(M, *args, *to, 0, P(ws), n, v4moe._stream()) == 0
        assert torch.equal(got, one)


@pytest.mark.parametrize("shape", [(1, 2048, 2048), (16, 256, 4096), (9, 64, 8), (40, 512, 1000), (5, 33, 1048), (3, 100, 2056),
                                   (16, 4000, 1096), (4300, 16, 1200)], ids=str)
def test_linear_of_few_rows(shape):
    """bf16 rows at 16-byte addresses are quantised inside the product; others beforehand: the same bits."""
    M, N, K = shape
    x = source(7, M, K, torch.bfloat16)
    x[0, 0] = 1e-30
    w = v4moe.fp8_weights(source(8, N, K, torch.float32))
    moved = torch.empty(M * K + 1, dtype=torch.bfloat16, device=DEV)[1:].view(M, K).copy_(x)
    assert torch.equal(v4moe.fp8_linear(x, w), v4moe.fp8_linear(moved, w))
    tiny = (x.float() * 1e-33).to(torch.bfloat16)      # scales down to subnormal numbers
    assert torch.equal(v4moe.fp8_linear(tiny, w), v4moe.fp8_linear(moved.copy_(tiny), w))
    x[0, K - 1] = math.inf
    y = v4moe.fp8_linear(x, w)
    assert bool(y[0].isnan().all()) and not y[1:].isnan().any()


def test_gradient_against_differences():
    """L = <dy, x W^T> is linear in x and in W, so its differences are exact; what E4M3 rounds off
    is at most 2^-4 of each operand's elements, independent of each other: 2^-4 in the 2-norm for each operand."""
    M, N, K = 64, 96, 160
    x, w0, dy = (torch.randn(*s, device=DEV, dtype=torch.float64) for s in ((M, K), (N, K), (M, N)))
    w = v4moe.fp8_weights(w0.float())
    dx, dw = v4moe.fp8_linear_backward(x.float(), dy.float(), w)
    loss = lambda x, w: (dy * (x @ w.t())).sum()  # noqa: E731
    h = 1e-3

    def differences(f, t):
        out = torch.empty_like(t)
        for i in range(0, t.numel(), 37):
            e = torch.zeros_like(t).view(-1)
            e[i] = h
            out.view(-1)[i] = (f(t + e.view_as(t)) - f(t - e.view_as(t))) / (2 * h)
        return out.view(-1)[::37]

    for got, want in ((dx, differences(lambda t: loss(t, w0), x)), (dw, differences(lambda t: loss(x, t), w0))):
        d = got.double().reshape(-1)[::37] - want
        assert float(d.norm() / want.norm()) <= 2 * 2.0 ** -4


def test_streams():
    x = torch.randn(300, 512, device=DEV)
    w0 = torch.randn(400, 512, device=DEV)
    w = v4moe.fp8_weights(w0)
    y = v4moe.fp8_linear(x, w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y2 = v4moe.fp8_linear(x, v4moe.fp8_weights(w0))
    s.synchronize()
    assert torch.equal(y, y2)


def test_graph():
    """A captured forward and backward replays to the eager results."""
    x, dy = torch.randn(70, 512, device=DEV), torch.randn(70, 300, device=DEV)
    w = v4moe.fp8_weights(torch.randn(300, 512, device=DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        v4moe.fp8_linear(x, w)
        v4moe.fp8_linear_backward(x, dy, w)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = v4moe.fp8_linear(x, w)
        dx, dw = v4moe.fp8_linear_backward(x, dy, w)
    for i in range(3):
        x.copy_(torch.randn(70, 512, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        ey = v4moe.fp8_linear(x, w)
        edx, edw = v4moe.fp8_linear_backward(x, dy, w)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(dx, edx) and torch.equal(dw, edw)
