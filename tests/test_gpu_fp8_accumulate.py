"""moe_fp8_gemm and the weight gradient added to what a matrix holds.

Bit for bit: the fp32 result does not depend on the variant or on the type of C, so adding it to an old value is
one fp32 addition and, for a bf16 C, one rounding of that sum."""
import pytest
import torch

from fp4_weight_grouped_amd import v4moe
from test_gpu_fp8 import DEV, _float32, operand, source  # noqa: F401

pytestmark = pytest.mark.gpu

# the variant of few rows, each tile, ragged edges
SHAPES = [(1, 64, 128), (3, 17, 144), (16, 300, 2048), (17, 129, 256), (65, 1000, 384), (200, 384, 128), (700, 1030, 256),
          (1100, 900, 384), (2050, 1300, 160), (70, 2200, 1200), (1000, 3100, 144), (4100, 4000, 400)]


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gemm(shape, type, rows):
    M, N, K = shape
    a, sa = operand(M, M, K, 0, True)
    b, sb = operand(N + 7, N, K, 0, True)
    sa, sb = sa.t().contiguous(), sb.t().contiguous() if rows else sb[::128].contiguous()
    new = v4moe.fp8_gemm(a, sa, b, sb, rows, out=torch.empty(M, N, device=DEV))
    g = torch.Generator(device=DEV).manual_seed(K)
    for pad, at in ((0, 0), (3, 1)):
        buf = (torch.randn(M, N + pad, generator=g, device=DEV) * new.std()).to(type)
        old = buf.clone()
        v4moe.fp8_gemm(a, sa, b, sb, rows, out=buf[:, at:at + N], accumulate=True)
        assert torch.equal(buf[:, at:at + N], (old[:, at:at + N].float() + new).to(type))
        assert torch.equal(buf[:, :at], old[:, :at]) and torch.equal(buf[:, at + N:], old[:, at + N:])


@pytest.mark.parametrize("type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 128, 256), (9, 77, 130), (300, 1000, 900), (1237, 999, 1001), (2100, 1500, 3000)], ids=str)
def test_weight_gradient(shape, type):
    M, N, K = shape
    x, dy = source(5, M, K, torch.bfloat16), source(6, M, N, torch.bfloat16)
    w = v4moe.fp8_weights(source(7, N, K, torch.float32))
    dx0, new = v4moe.fp8_linear_backward(x, dy, w, dw=torch.empty(N, K, device=DEV))
    old = (torch.randn(N, K, device=DEV) * new.std()).to(type)
    dx, dw = v4moe.fp8_linear_backward(x, dy, w, dw=old.clone(), accumulate=True)
    assert torch.equal(dx, dx0) and torch.equal(dw, (old.float() + new).to(type))
    # many small contributions: each rounds the sum once, so a constant one adds up to within half a bf16 step each
    dw = torch.zeros(N, K, dtype=type, device=DEV)
    want = torch.zeros(N, K, device=DEV)
    for _ in range(4):
        v4moe.fp8_linear_backward(x, dy, w, dw=dw, accumulate=True)
        want = (want + new).to(type).float()
    assert torch.equal(dw.float(), want)


@pytest.mark.parametrize("type", [torch.bfloat16, torch.float32])
def test_weight_gradient_of_no_rows(type):
    """Left alone, in every bit, where it accumulates; zero otherwise."""
    w = v4moe.fp8_weights(torch.randn(33, 50, device=DEV))
    x, dy = torch.zeros(0, 50, device=DEV), torch.zeros(0, 33, device=DEV)
    old = torch.randn(33, 50, device=DEV).to(type)
    old[::2] = -0.0
    old[1] = float("nan")
    bits = torch.int16 if type == torch.bfloat16 else torch.int32
    dw = old.clone()
    v4moe.fp8_linear_backward(x, dy, w, dw=dw, accumulate=True)
    assert torch.equal(dw.view(bits), old.view(bits))
    v4moe.fp8_linear_backward(x, dy, w, dw=dw)
    assert not dw.view(bits).any()
