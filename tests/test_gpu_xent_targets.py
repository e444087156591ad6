"""Gradients of the cross entropy where nearly all of them is the targets' own term.

d[t][v] = g_t (p[t][v] - [v = y_t]) enters the products in bf16.  Where the probabilities are spread over many columns,
d at the target is most of a gradient, and its rounding would be off by a whole bf16 step of it: what the rounding left
there is added again, so that it is off by 2^-16 of itself only.

Here the columns that no token aims at have weights close to zero: their share of the sums, and so of the bound, is
small, and a rounding of the targets' d alone would be past it.  Bounds: as of the other tests of these gradients
(logits off by ez, the log-sum-exp by el, sums in fp32), but for d at the target 2^-16 of itself in place of 2^-8, and
one more product of the sums for each token."""
import pytest
import torch

from fp4_weight_grouped_amd import v4moe

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _float32():
    old = torch.get_default_dtype()
    torch.set_default_dtype(F32)
    yield
    torch.set_default_dtype(old)


def rows(n, cols, pad, std):
    return torch.randn(n, cols + pad, device=DEV).mul_(std).to(BF16)[:, :cols]


def inputs(T, H, V, aimed, pad=0):
    """Targets among `aimed` columns of ordinary weights, every fifth token without one; weights of the others 2^-10 of that."""
    x, w = rows(T, H, pad, 1.0), rows(V, H, pad, H ** -0.5 * 2.0 ** -10)
    columns = torch.randperm(V, device=DEV)[:aimed]
    w[columns] = torch.randn(len(columns), H, device=DEV).mul_(H ** -0.5).to(BF16)
    y = columns[torch.randint(0, len(columns), (T,), device=DEV)]
    y[torch.arange(T, device=DEV) % 5 == 4] = -100
    return x, w, y


def reference(x, w, y, g):
    """(lse, (dx, its bound), (dw, its bound)) in 64 bits."""
    T, (V, H) = x.shape[0], w.shape
    k = torch.nonzero(y >= 0).flatten()
    a, b, t, n = x.double()[k], w.double(), y[k], len(k)
    at = torch.arange(n, device=DEV)
    z = a @ b.t()
    ez = ((H + 32) * 2.0 ** -23 * (a.abs() @ b.abs().t())).amax(dim=1)
    lse = torch.logsumexp(z, dim=1)
    el = ez + (z.amax(dim=1) - z.amin(dim=1) + 128 + V / 4096) * 2.0 ** -22 + lse.abs() * 2.0 ** -23
    p = (z - lse.unsqueeze(1)).exp()
    del z
    gk = g.double()[k].unsqueeze(1)
    err = gk.abs() * p * (ez + el + 2.0 ** -22).unsqueeze(1) * 1.01
    d = p
    d[at, t] -= 1.0
    d *= gk
    rounding = torch.full_like(d, 2.0 ** -8 + 2.0 ** -22)
    rounding[at, t] = 2.0 ** -16 + 2.0 ** -22
    err += d.abs() * rounding
    del rounding
    size = d.abs() + err

    def full(v, *shape):
        f = torch.zeros(T, *shape, dtype=torch.float64, device=DEV)
        f[k] = v
        return f

    dx = full(d @ b, H), full(err @ b.abs() + (V + 65) * 2.0 ** -23 * (size @ b.abs()), H)
    dw = d.t() @ a, err.t() @ a.abs() + (2 * n + 64) * 2.0 ** -23 * (size.t() @ a.abs())
    return full(lse).float(), dx, dw


def close(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


def test_many_tokens_in_either_tile():
    """Cases of more than 4096 tokens with a target, which dW's tiles take in turns, are of both tiles."""
    many = (12000, 40, 3000), (12000, 64, 700), (6000, 2056, 20000)
    tiles = {H: v4moe.lib().moe_linear_xent_tile(T, H, V, 2, 1) & 0xFFFF for T, H, V in many}
    assert tiles == {40: 128, 64: 128, 2056: 256}


# tokens, width, columns, columns aimed at: few tokens and many; targets of their own and one for all; a partial last
# tile; a vocabulary in several pieces; products of 128x128 tiles, both in one launch, and of 256x256; more than 4096 tokens
# with a target, all of them in one tile, too
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,V,aimed", [
    (12000, 40, 3000, 50), (12000, 64, 700, 1), (6000, 2056, 20000, 300), (6000, 2056, 20000, 1),
    (1, 64, 5000, 1), (3, 40, 5000, 3), (40, 264, 5003, 30), (300, 72, 5000, 100), (300, 104, 5000, 1), (700, 1001, 9001, 200),
    (1500, 136, 9000, 1000), (4100, 32, 66000, 300), (5000, 64, 20011, 1), (700, 2048, 16500, 100), (2000, 1024, 40000, 2),
])
@pytest.mark.parametrize("pad", [0, 3])
def test_the_targets_keep_their_digits(T, H, V, aimed, pad):
    torch.manual_seed(T + H + V + pad)
    x, w, y = inputs(T, H, V, aimed, pad)
    g = (torch.rand(T, device=DEV) + 0.1) / T
    lse, (dx, dx_bound), (dw, dw_bound) = reference(x, w, y, g)
    for t in (BF16, F32):
        gx, gw = torch.empty(T, H, dtype=t, device=DEV), torch.empty(V, H, dtype=t, device=DEV)
        v4moe.linear_xent_backward(x, w, y, lse, g, dx=gx, dw=gw)
        close(gx, dx, dx_bound, "dx")
        close(gw, dw, dw_bound, "dw")
    before = torch.randn(V, H, device=DEV) / T
    after = before.clone()
    v4moe.linear_xent_backward(x, w, y, lse, g, dw=after, accumulate=True)
    close(after, before.double() + dw, dw_bound + 2.0 ** -23 * (before.double().abs() + dw.abs() + dw_bound), "dw added to")


@pytest.mark.gpu
def test_rounded_once():
    """The gradients of either type come of the same sums, and repeat themselves."""
    torch.manual_seed(0)
    x, w, y = inputs(900, 200, 5000, 40)
    g = torch.rand(900, device=DEV)
    _, lse = v4moe.linear_xent(x, w, y)
    want = v4moe.linear_xent_backward(x, w, y, lse, g, dx=torch.empty(900, 200, device=DEV), dw=torch.empty(5000, 200, device=DEV))
    for _ in range(3):
        got = v4moe.linear_xent_backward(x, w, y, lse, g)
        assert all(torch.equal(p, q.to(BF16)) for p, q in zip(got, want))
