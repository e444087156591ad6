"""moe_clip_grads where the joint norm or the coefficient leaves fp32's normal numbers.

Bars as in test_gpu_clip.py: 3 * 2^-23 relative for fp32 and 2^-8 for bf16, plus half of the type's smallest
step where a result is no normal number (bf16 and fp32 share the exponent's range; bf16's steps are 2^16 as wide)."""
import math

import pytest
import torch

from fp4_weight_grouped_amd import v4moe
from test_gpu_clip import DEV, _float32  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = torch.finfo(torch.float32).max
CASES = [(3e38, 64, 1.0), (3e38, 100_003, 1.0), (3e38, 1000, 3e38), (FLT_MAX, 5, FLT_MAX), (1e30, 1000, 1e-12),
         (1e38, 10, 1e-30), (3e38, 70_000, 1e-37), (1e-3, 1000, 1e-45), (3e38, 64, 0.0), (3e38, 64, math.inf)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("size,n,max_norm", CASES)
def test_range(size, n, max_norm, in_place):
    sign = torch.randn(n + 1, device=DEV).sign()[1:]              # a view off 16 bytes
    grads = [sign * size, (sign[: n // 2 + 1] * (size / 3)).to(torch.bfloat16), torch.zeros(3, device=DEV)]
    keep = [g.clone() for g in grads]
    out = None if in_place else [torch.full_like(g, 7.0) for g in grads]
    norm = v4moe.clip_grads(grads, max_norm, out=out)
    limit = float(torch.tensor(max_norm, dtype=torch.float32))
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in keep))
    if ref > FLT_MAX * (1 + 2.0 ** -24):
        assert math.isinf(float(norm))
    else:
        assert abs(float(norm) - ref) <= ref * 2.0 ** -23
    c = limit / ref if ref > limit else 1.0
    for k, o in zip(keep, grads if in_place else out):
        want = k.double() * c
        bf16 = k.dtype == torch.bfloat16
        tol = want.abs() * (2.0 ** -8 if bf16 else 3 * 2.0 ** -23) + (2.0 ** -134 if bf16 else 2.0 ** -150)
        assert bool(((o.double() - want).abs() <= tol).all()), float(((o.double() - want).abs() / tol).max())


def test_infinite_gradients_are_still_left_alone():
    """An infinity among gradients is not a norm beyond fp32's range: nothing is scaled."""
    for bad in (math.inf, math.nan):
        g = [torch.full((1000,), 3e38, device=DEV), torch.ones(50, device=DEV)]
        g[1][7] = bad
        keep = [x.clone() for x in g]
        assert not math.isfinite(float(v4moe.clip_grads(g, 0.5)))
        for o, k in zip(g, keep):
            assert torch.equal(torch.nan_to_num(o, nan=123.0), torch.nan_to_num(k, nan=123.0))
