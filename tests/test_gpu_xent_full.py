"""Gradients of the cross entropy with all of the logits' gradient kept to 16 bits (full), against the formula in 64 bits.

Bounds: as of the other tests of these gradients (a logit off by ez = (H + 32) 2^-23 of its products' magnitudes, the
log-sum-exp by el = ez + (range + 128 + V / 4096) 2^-22, sums in fp32), but every d is off by 2^-16 of itself where one
bf16 number would be by 2^-8, and the sums have two products for each."""
import math

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _float32():
    old = torch.get_default_dtype()
    torch.set_default_dtype(F32)
    yield
    torch.set_default_dtype(old)


def rows(n, cols, pad=0, std=1.0):
    return torch.randn(n, cols + pad, device=DEV).mul_(std).to(BF16)[:, :cols]


def close(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


class Formula:
    def __init__(self, x, w, y, g):
        T, (V, H) = x.shape[0], w.shape
        k = self.rows = torch.nonzero((y >= 0) & (y < V)).flatten()
        a, b, n = x.double()[k], w.double(), len(k)
        at = torch.arange(n, device=DEV)
        z = a @ b.t()
        ez = ((H + 32) * 2.0 ** -23 * (a.abs() @ b.abs().t())).amax(dim=1)
        lse = torch.logsumexp(z, dim=1)
        el = ez + (z.amax(dim=1) - z.amin(dim=1) + 128 + V / 4096) * 2.0 ** -22 + lse.abs() * 2.0 ** -23
        d = torch.softmax(z, dim=1)
        del z
        gk = g.double()[k].unsqueeze(1)
        err = gk.abs() * d * (ez + el + 2.0 ** -22).unsqueeze(1) * 1.01
        d[at, y[k]] -= 1.0
        d *= gk
        err += d.abs() * (2.0 ** -16 + 2.0 ** -22)
        size = d.abs() + err
        self.dx, self.dx_bound, self.lse = (torch.zeros(T, s, dtype=torch.float64, device=DEV) for s in (H, H, 1))
        self.lse[k, 0] = lse
        self.lse = self.lse[:, 0].float()
        self.dx[k], self.dx_bound[k] = d @ b, err @ b.abs() + (2 * V + 64) * 2.0 ** -23 * (size @ b.abs())
        self.dw, self.dw_size = d.t() @ a, size.t() @ a.abs()
        self.dw_bound = err.t() @ a.abs() + (2 * n + 64) * 2.0 ** -23 * self.dw_size


# few tokens and many, every tile, partial last tiles and slices, one piece of the vocabulary and several, the smallest
# pieces; logits whose probabilities are spread and such that a few columns have them all
@pytest.mark.parametrize("T,H,V,pad", [(1, 64, 300, 0), (2, 1, 2, 0), (5, 8, 1, 0), (20, 72, 1000, 3), (60, 136, 5000, 0), (300, 257, 4099, 3),
                                       (700, 64, 20000, 0), (1500, 136, 9000, 8), (2000, 2056, 300, 0), (1000, 2056, 33000, 0),
                                       (4100, 32, 66000, 0), (4100, 1025, 40001, 0)])
@pytest.mark.parametrize("std", [0.5, 5.0])
def test_gradients(T, H, V, pad, std):
    torch.manual_seed(T + H + V)
    x, w = rows(T, H, pad), rows(V, H, pad, std * H ** -0.5)
    y = torch.randint(0, V, (T,), device=DEV)
    y[torch.arange(T, device=DEV) % 4 == 3] = -100
    g = torch.randn(T, device=DEV) / T
    r = Formula(x, w, y, g)
    for t in (F32, BF16):
        dx, dw = torch.full((T, H + pad), 7.0, dtype=t, device=DEV), torch.full((V, H + pad), 7.0, dtype=t, device=DEV)
        v4moe.linear_xent_backward(x, w, y, r.lse, g, dx=dx[:, :H], dw=dw[:, :H], full=True)
        close(dx[:, :H], r.dx, r.dx_bound, "dx")
        close(dw[:, :H], r.dw, r.dw_bound, "dw")
        assert bool((dx[:, H:] == 7.0).all()) and bool((dw[:, H:] == 7.0).all())
        none = torch.ones(T, dtype=torch.bool, device=DEV)
        none[r.rows] = False
        assert not bool(dx[:, :H][none].any())
        before = torch.randn(V, H, device=DEV).to(t) / T
        after = before.clone()
        v4moe.linear_xent_backward(x, w, y, r.lse, g, dw=after, accumulate=True, full=True)
        close(after, before.double() + r.dw, r.dw_bound + 2.0 ** -23 * (before.double().abs() + r.dw_size), "dw added to")
    # each alone
    dx, none = v4moe.linear_xent_backward(x, w, y, r.lse, g, dx=torch.empty(T, H, device=DEV), need_dw=False, full=True)
    close(dx, r.dx, r.dx_bound, "dx alone")
    none, alone = v4moe.linear_xent_backward(x, w, y, r.lse, g, need_dx=False, full=True)
    assert none is None and torch.equal(alone, dw[:, :H])


def test_many_batches_add_up():
    """Gradients of a head from many batches, added in place, keep the digits of one batch."""
    torch.manual_seed(1)
    V, H, n, T = 3000, 200, 12, 150
    w, held, want, bound = rows(V, H, 0, 3 * H ** -0.5), torch.zeros(V, H, device=DEV), 0, 0
    for _ in range(n):
        x, y, g = rows(T, H), torch.randint(0, V, (T,), device=DEV), torch.rand(T, device=DEV) / T
        r = Formula(x, w, y, g)
        v4moe.linear_xent_backward(x, w, y, r.lse, g, dw=held, accumulate=True, full=True, need_dx=False)
        want, bound = want + r.dw, bound + r.dw_bound + n * 2.0 ** -23 * r.dw_size
    close(held, want, bound, "dw")


def test_masked_rows_infinities_and_nan():
    torch.manual_seed(2)
    T, H, V = 150, 96, 1000
    x, w, y = rows(T, H), rows(V, H, 0, 1.5 * H ** -0.5), torch.randint(0, V, (T,), device=DEV)
    y[::3] = -100
    g = torch.rand(T, device=DEV)
    r = Formula(x, w, y, g)
    off = y < 0
    x[off], r.lse[off], g[off] = math.nan, math.nan, math.inf
    dx, dw = v4moe.linear_xent_backward(x, w, y, r.lse, g, full=True)
    close(dx, r.dx, r.dx_bound, "dx")
    close(dw, r.dw, r.dw_bound, "dw")
    bad = int(r.rows[3])
    g[bad] = math.inf                                    # stays with its token
    dx, _ = v4moe.linear_xent_backward(x, w, y, r.lse, g, full=True)
    keep = torch.arange(T, device=DEV) != bad
    close(dx[keep], r.dx[keep], r.dx_bound[keep], "dx")
    assert not bool(dx[bad].isfinite().any())
    y[:] = -100                                          # no target at all
    held = torch.randn(V, H, device=DEV)
    same = held.clone()
    dx, dw = v4moe.linear_xent_backward(x, w, y, r.lse, g, full=True)
    assert not bool(dx.any()) and not bool(dw.any())
    v4moe.linear_xent_backward(x, w, y, r.lse, g, dw=held, accumulate=True, full=True)
    assert torch.equal(held, same)
    # no tokens
    e = x[:0]
    dx, dw = v4moe.linear_xent_backward(e, w, y[:0], g[:0], g[:0], full=True)
    assert dx.shape == (0, H) and not bool(dw.any())
    v4moe.linear_xent_backward(e, w, y[:0], g[:0], g[:0], dw=held, accumulate=True, full=True)
    assert torch.equal(held, same)


def test_captured_and_repeated():
    """Captured beside a call in bf16, whose workspace is another; replayed with other inputs; the same bits each time."""
    torch.manual_seed(3)
    T, H, V = 600, 101, 3001
    x, w, y, g = rows(T, H), rows(V, H, 0, 2 * H ** -0.5), torch.randint(-900, V, (T,), device=DEV), torch.rand(T, device=DEV)

    def step():
        _, lse = v4moe.linear_xent(x, w, y)
        return *v4moe.linear_xent_backward(x, w, y, lse, g, full=True), *v4moe.linear_xent_backward(x, w, y, lse, g)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        x.copy_(torch.randn_like(x))
        y.copy_(torch.randint(-900, V, (T,), device=DEV))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
