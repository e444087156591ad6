"""moe_clip_grads against a plain 64-bit implementation.

Bars.  norm: an fp64 sum rounded once to fp32, 2^-23 relative.  out: the
coefficient is one fp32 division of that norm and the product one more rounding:
3 * 2^-23 relative for fp32, 2^-8 for bf16 (values are normal numbers)."""
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


def make(seed, sizes, bf16=()):
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        at = i % 5                       # views that begin inside a buffer, at every alignment
        t = torch.bfloat16 if i in bf16 else torch.float32
        b = torch.randn(n + at, generator=g, device=DEV).to(t) * (1 + i)
        out.append(b[at:])
    return out


def check(grads, max_norm, got, norm):
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - ref) <= ref * 2.0 ** -23
    c = max_norm / ref if ref > max_norm else 1.0
    for g, o in zip(grads, got):
        want = g.double() * c
        tol = want.abs() * (2.0 ** -8 if g.dtype == torch.bfloat16 else 3 * 2.0 ** -23)
        assert o.dtype == g.dtype and bool(((o.double() - want).abs() <= tol).all())


SIZES = [[1], [5, 0, 3], [16384], [16383, 16385, 1], [100003, 7, 1 << 20, 33], [257] * 130, [3] * 96 + [5] * 97]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("max_norm", [0.0, 0.25, 1e9, math.inf])
def test_out_of_place_and_in_place(sizes, max_norm):
    bf16 = {i for i in range(len(sizes)) if i % 3 == 1}
    grads = make(1, sizes, bf16)
    keep = [g.clone() for g in grads]
    for shift in (0, 1):                 # out aligned as the gradient, and differently
        outs = [torch.full((g.numel() + 8,), 7.0, dtype=g.dtype, device=DEV) for g in grads]
        view = [o[(i + shift) % 5:][:g.numel()] for i, (o, g) in enumerate(zip(outs, grads))]
        norm = v4moe.clip_grads(grads, max_norm, out=view)
        check(keep, max_norm, view, norm)
        assert all(torch.equal(g, k) for g, k in zip(grads, keep))
        for i, (o, g) in enumerate(zip(outs, grads)):      # nothing beside the view is written
            at = (i + shift) % 5
            assert bool((o[:at] == 7).all()) and bool((o[at + g.numel():] == 7).all())
    norm2 = v4moe.clip_grads(grads, max_norm)
    assert torch.equal(norm, norm2)
    check(keep, max_norm, grads, norm2)
    if float(norm) <= max_norm:
        assert all(torch.equal(g, k) for g, k in zip(grads, keep))


def test_magnitudes():
    """fp32's whole range: squares neither overflow nor vanish."""
    for v in (1e30, 1e-30, 1e-40):
        g = [torch.full((1000,), v, device=DEV), torch.full((24,), v, device=DEV)]
        norm = v4moe.clip_grads(g, math.inf)
        assert abs(float(norm) / (v * 32) - 1) < 1e-4


def test_not_finite():
    for bad in (math.inf, -math.inf, math.nan):
        g = make(2, [1000, 50], {1})
        g[1][7] = bad
        keep = [x.clone() for x in g]
        out = [torch.empty_like(x) for x in g]
        norm = v4moe.clip_grads(g, 0.5, out=out)
        assert not math.isfinite(float(norm))
        for o, k in zip(out, keep):
            assert torch.equal(torch.nan_to_num(o, nan=123.0), torch.nan_to_num(k, nan=123.0))
        v4moe.clip_grads(g, 0.5)
        for o, k in zip(g, keep):
            assert torch.equal(torch.nan_to_num(o, nan=123.0), torch.nan_to_num(k, nan=123.0))


def test_zero_gradients_and_streams():
    g = [torch.zeros(1000, device=DEV)]
    assert float(v4moe.clip_grads(g, 0.0)) == 0.0 and float(g[0].abs().max()) == 0.0
    s = torch.cuda.Stream()
    a = make(3, [50000, 123], {1})
    b = [x.clone() for x in a]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        n1 = v4moe.clip_grads(a, 0.5)
    s.synchronize()
    n2 = v4moe.clip_grads(b, 0.5)
    assert torch.equal(n1, n2) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_repeatable():
    g = make(4, [3_000_000, 70_001, 12], {1})
    first = v4moe.clip_grads(g, math.inf)
    for _ in range(5):
        assert torch.equal(first, v4moe.clip_grads(g, math.inf))


def test_more_than_2_to_31_elements():
    """Offsets past 32 bits, in one tensor."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[-1] = 3.0
    g[1 << 31] = 4.0
    norm = v4moe.clip_grads([g], 2.5)
    assert float(norm) == 5.0 and float(g[-1]) == 1.5 and float(g[1 << 31]) == 2.0
    assert float(g[:1000].abs().max()) == 0.0
