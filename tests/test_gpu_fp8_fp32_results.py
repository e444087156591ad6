"""fp32 results of the FP8 products next to those of the same codes and scales multiplied in fp32.

The matrix instruction aligns a chunk's 128 products to the largest and drops what lies far below, so an fp32 result
is not as exact as fp32 sums of the products: 1.3e-5 in the 2-norm was measured for codes of normal numbers, and twice
that is the bar (fp32 products of the same values: printed beside it).  A bf16 result has 1.7e-3 of its own rounding (2^-9 / sqrt(3) and less), which hides it: the bar there
is 2^-9."""
import pytest
import torch

from fp4_weight_grouped_amd import v4moe
from test_gpu_fp8 import DEV, _float32, values  # noqa: F401

pytestmark = pytest.mark.gpu
FP32, BF16 = 2.7e-5, 2.0 ** -9


def spread(q, s, along):
    """Values of codes q with scales s [chunks][rows], chunks of 128 of the columns."""
    return values(q) * s.t().double()[:, torch.arange(along, device=DEV) // 128]


@pytest.mark.parametrize("M,N,K", [(16, 512, 2048), (300, 500, 1000), (1024, 1024, 4096)])
def test_error(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(M)
    x, dy, w0 = (torch.randn(*s, generator=g, device=DEV) for s in ((M, K), (M, N), (N, K)))
    w = v4moe.fp8_weights(w0)
    qx, sx, qxt, sxt = v4moe.fp8_quantize(x, True, True)
    _, _, qyt, syt = v4moe.fp8_quantize(dy, True, True)
    blk = w.blk.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    W, X = values(w.q[:, :K]) * blk, spread(qx[:, :K], sx, K)
    XT, YT = spread(qxt[:, :M], sxt, M), spread(qyt[:, :M], syt, M)
    cases = [(lambda t: v4moe.fp8_linear(x, w, out=torch.empty(M, N, dtype=t, device=DEV)), X, W),
             (lambda t: v4moe.fp8_linear_backward(x, dy, w, dw=torch.empty(N, K, dtype=t, device=DEV))[1], YT, XT)]
    for own, a, b in cases:
        ref = a @ b.t()
        error = lambda r: float((r.double() - ref).norm() / ref.norm())  # noqa: E731
        own32, plain32, own16 = error(own(torch.float32)), error(a.float() @ b.float().t()), error(own(torch.bfloat16))
        print(f"{M}x{N}x{K}: fp32 {own32:.2e} (fp32 products {plain32:.2e}), bf16 {own16:.2e}")
        assert own32 <= FP32 and own16 <= BF16
