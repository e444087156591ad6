"""Softmax cross entropy over a vocabulary against the formula in 64 bits.

Bounds.  A logit is one chain of fp32 additions of exact bf16 products, 32 terms to an
instruction: off by at most ez = (H + 32) 2^-23 times the sum of its products' magnitudes.
A shift of every logit by at most ez shifts the log-sum-exp by at most that; its own sum
adds the exponentials' errors (the exponent's product is rounded: |z - max| 2^-24 of each
term, and 2^-22 for the instruction) and at most 64 + V / 4096 additions in a row: el =
ez + (range + 128 + V / 4096) 2^-22, and half a step of the result.  A probability is then
off by ez + el of itself, its gradient is rounded to bf16 (2^-8), and the products' sums
as above."""
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


def rows(n, cols, pad=0, std=1.0, at=0):
    buf = torch.randn(n * (cols + pad) + at, device=DEV).mul_(std).to(BF16)
    return buf[at:].view(n, cols + pad)[:, :cols]


def inputs(T, H, V, pad=0, none=0.2, std=1.5, at=0):
    x, w = rows(T, H, pad, at=at), rows(V, H, pad, std * H ** -0.5)
    y = torch.randint(0, V, (T,), device=DEV)
    off = torch.rand(T, device=DEV) < none
    y[off] = torch.tensor([-100, -1, V, 2 ** 40], device=DEV)[torch.arange(T, device=DEV) % 4][off]
    return x, w, y


class Reference:
    """The formula in 64 bits over the tokens with a target, and the bounds above."""

    def __init__(self, x, w, y, g=None):
        T, (V, H) = x.shape[0], w.shape
        self.kept = (y >= 0) & (y < V)
        k = self.rows = torch.nonzero(self.kept).flatten()
        a, b, t = x.double()[k], w.double(), y[k]
        z, n = a @ b.t(), len(k)
        ez = (H + 32) * 2.0 ** -23 * (a.abs() @ b.abs().t())
        ez = ez.amax(dim=1) if n else torch.zeros(0, dtype=torch.float64, device=DEV)
        lse = torch.logsumexp(z, dim=1)
        reach = z.amax(dim=1) - z.amin(dim=1) if n else ez
        el = ez + (reach + 128 + V / 4096) * 2.0 ** -22
        at = torch.arange(n, device=DEV)

        def full(v, *shape):
            f = torch.zeros(T, *shape, dtype=torch.float64, device=DEV)
            f[k] = v
            return f

        loss = lse - z[at, t]
        self.lse, self.lse_bound = full(lse), full(el + lse.abs() * 2.0 ** -23)
        self.loss, self.loss_bound = full(loss), full(ez + el + (lse.abs() + loss.abs()) * 2.0 ** -23)
        if g is None:
            return
        p = torch.softmax(z, dim=1)
        hot = torch.zeros_like(p)
        hot[at, t] = 1.0
        gk = g.double()[k].unsqueeze(1)
        d = gk * (p - hot)
        err = gk.abs() * p * (ez + self.lse_bound[k] + 2.0 ** -22).unsqueeze(1) * 1.01 + d.abs() * (2.0 ** -8 + 2.0 ** -22)
        self.dx, self.dw = full(d @ b, H), d.t() @ a
        size = d.abs() + err
        self.dx_bound = full(err @ b.abs() + (V + 64) * 2.0 ** -23 * (size @ b.abs()), H)
        self.dw_bound = err.t() @ a.abs() + (n + 64) * 2.0 ** -23 * (size.t() @ a.abs())
        self.dw_size = size.t() @ a.abs()


def close(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


# T, H, V: every tile (by T, and by T x V), one token, one column, a partial last group of 64 columns, contractions of
# less than a step and of a partial last one, a vocabulary in several pieces
SHAPES = [
    (1, 64, 300), (1, 8, 1), (2, 1, 2), (16, 72, 64), (17, 64, 65), (32, 100, 1000), (33, 128, 63), (64, 264, 513),
    (65, 40, 4099), (200, 512, 777), (300, 104, 1031), (700, 64, 20000), (1500, 136, 9000), (4100, 32, 66000), (5, 4096, 130),
]


# rows alone, inside wider aligned ones, inside wider odd ones (the largest in one layout)
@pytest.mark.parametrize("T,H,V,pad", [(*shape, pad) for shape in SHAPES for pad in (0, 8, 3) if shape[0] < 1000 or pad == 0])
def test_loss_and_gradients(T, H, V, pad):
    torch.manual_seed(T + H + V + pad)
    x, w, y = inputs(T, H, V, pad)
    g = torch.randn(T, device=DEV) / T
    r = Reference(x, w, y, g)
    loss, lse = v4moe.linear_xent(x, w, y)
    assert loss.dtype == lse.dtype == F32
    close(lse, r.lse, r.lse_bound, "lse")
    close(loss, r.loss, r.loss_bound, "loss")
    assert not bool(loss[~r.kept].any()) and not bool(lse[~r.kept].any())
    for t in (BF16, F32):
        dx = torch.full((T, H + pad), 7.0, dtype=t, device=DEV)
        dw = torch.full((V, H + pad), 7.0, dtype=t, device=DEV)
        v4moe.linear_xent_backward(x, w, y, lse, g, dx=dx[:, :H], dw=dw[:, :H])
        close(dx[:, :H], r.dx, r.dx_bound, "dx")
        close(dw[:, :H], r.dw, r.dw_bound, "dw")
        assert bool((dx[:, H:] == 7.0).all()) and bool((dw[:, H:] == 7.0).all())
        assert not bool(dx[:, :H][~r.kept].any())
        before = torch.randn(V, H, device=DEV).to(t) / T
        after = before.clone()
        v4moe.linear_xent_backward(x, w, y, lse, g, dw=after, accumulate=True)
        # (one more addition, of the sum to what was there)
        close(after, before.double() + r.dw, r.dw_bound + 2.0 ** -23 * (before.double().abs() + r.dw_size), "dw added to")


@pytest.mark.parametrize("count", [1, 16, 30, 60, 150, 500])
def test_a_token_does_not_depend_on_the_others(count):
    """Loss and log-sum-exp in every bit, whichever tile the batch has, and wherever the tokens without a target are."""
    torch.manual_seed(count)
    x, w, y = inputs(600, 200, 3001, none=0.0)
    loss, lse = v4moe.linear_xent(x, w, y)
    a, b = v4moe.linear_xent(x[:count], w, y[:count])
    assert torch.equal(a, loss[:count]) and torch.equal(b, lse[:count])
    off = torch.rand(600, device=DEV) < 0.5
    c, d = v4moe.linear_xent(x, w, torch.where(off, -100, y))
    assert torch.equal(c[~off], loss[~off]) and torch.equal(d[~off], lse[~off])


def test_determinism():
    torch.manual_seed(0)
    x, w, y = inputs(333, 320, 5000)
    g = torch.rand(333, device=DEV)
    loss, lse = v4moe.linear_xent(x, w, y)
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, g)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(v4moe.linear_xent(x, w, y), (loss, lse)))
        assert all(torch.equal(a, b) for a, b in zip(v4moe.linear_xent_backward(x, w, y, lse, g), (dx, dw)))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_no_token_with_a_target(T):
    torch.manual_seed(T)
    x, w, y = inputs(T, 64, 100)
    y[:] = -100
    x[:] = math.nan
    loss, lse = v4moe.linear_xent(x, w, y)
    assert not bool(loss.any()) and not bool(lse.any())
    before = torch.randn(100, 64, device=DEV)
    after = before.clone()
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, torch.ones(T, device=DEV))
    assert not bool(dx.any()) and not bool(dw.any()) and not bool(dw.isnan().any())
    v4moe.linear_xent_backward(x, w, y, lse, torch.ones(T, device=DEV), dw=after, accumulate=True)
    assert torch.equal(before, after)


def test_rows_without_a_target_hold_anything():
    """NaN and infinities in x, lse and dloss of tokens without a target reach nothing."""
    torch.manual_seed(1)
    T, H, V = 150, 96, 1000
    x, w, y = inputs(T, H, V, none=0.3)
    g = torch.rand(T, device=DEV)
    r = Reference(x, w, y, g)
    x[~r.kept] = torch.tensor([math.nan, math.inf, -math.inf, 3e38], device=DEV).to(BF16)[torch.arange(H, device=DEV) % 4]
    loss, lse = v4moe.linear_xent(x, w, y)
    close(loss, r.loss, r.loss_bound, "loss")
    lse[~r.kept], g[~r.kept] = math.nan, math.inf
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, g)
    close(dx, r.dx, r.dx_bound, "dx")
    close(dw, r.dw, r.dw_bound, "dw")


def test_a_token_of_no_number_keeps_to_itself():
    torch.manual_seed(2)
    x, w, y = inputs(100, 64, 500, none=0.0)
    clean, _ = v4moe.linear_xent(x, w, y)
    x[7] = math.nan
    loss, lse = v4moe.linear_xent(x, w, y)
    assert bool(loss[7].isnan()) and bool(lse[7].isnan())
    keep = torch.arange(100, device=DEV) != 7
    assert torch.equal(loss[keep], clean[keep])
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, torch.ones(100, device=DEV))
    assert bool(dx[7].isnan().all()) and not bool(dx[keep].isnan().any()) and bool(dw.isnan().all())
    # a gradient that is infinite does not take the others' with it
    x, w, y = inputs(100, 64, 500, none=0.0)
    _, lse = v4moe.linear_xent(x, w, y)
    g = torch.rand(100, device=DEV)
    r = Reference(x, w, y, g)
    g[7] = math.inf
    dx, _ = v4moe.linear_xent_backward(x, w, y, lse, g)
    close(dx[keep], r.dx[keep], r.dx_bound[keep], "dx")
    assert not bool(dx[7].isfinite().any())


@pytest.mark.parametrize("big", [30.0, 3000.0])
def test_logits_far_apart(big):
    """Nothing overflows where the logits reach far: the largest is taken off first."""
    torch.manual_seed(3)
    T, H, V = 70, 64, 900
    x, w, y = inputs(T, H, V, none=0.1, std=big)
    g = torch.rand(T, device=DEV)
    r = Reference(x, w, y, g)
    loss, lse = v4moe.linear_xent(x, w, y)
    close(lse, r.lse, r.lse_bound, "lse")
    close(loss, r.loss, r.loss_bound, "loss")
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, g)
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())


@pytest.mark.parametrize("value", [0.0, 1.0 / 300, 1e-38, 1e30])
def test_one_gradient_for_all(value):
    """A mean's gradients come expanded (stride 0); very small and large ones keep their digits."""
    torch.manual_seed(4)
    T, H, V = 130, 80, 700
    x, w, y = inputs(T, H, V)
    g = torch.full((), value, device=DEV).expand(T)
    _, lse = v4moe.linear_xent(x, w, y)
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, g, dx=torch.empty(T, H, device=DEV), dw=torch.empty(V, H, device=DEV))
    # the same as for 1, scaled in fp32
    ux, uw = v4moe.linear_xent_backward(x, w, y, lse, torch.ones(T, device=DEV), dx=torch.empty(T, H, device=DEV),
                                        dw=torch.empty(V, H, device=DEV))
    if value == 0.0:
        assert not bool(dx.any()) and not bool(dw.any())
    else:
        s = torch.full((), value, device=DEV)
        assert torch.equal(dx, ux * s) and torch.equal(dw, uw * s)
    wide = torch.full((T, 3), value, device=DEV)
    a, b = v4moe.linear_xent_backward(x, w, y, lse, wide[:, 1])
    assert torch.equal(a, dx.to(BF16)) and torch.equal(b, dw.to(BF16))


def test_gradients_against_differences():
    """(L(x + h) - L(x - h)) / 2 = <dx, h> + O(h^3), L in 64 bits."""
    torch.manual_seed(5)
    T, H, V = 12, 32, 90
    x, w, y = inputs(T, H, V, none=0.2)
    g = torch.rand(T, device=DEV)
    _, lse = v4moe.linear_xent(x, w, y)
    dx, dw = v4moe.linear_xent_backward(x, w, y, lse, g, dx=torch.empty(T, H, device=DEV), dw=torch.empty(V, H, device=DEV))
    r = Reference(x, w, y, g)

    def L(a, b):
        z, k = a @ b.t(), r.rows
        return float((g.double()[k] * (torch.logsumexp(z[k], dim=1) - z[k, y[k]])).sum())

    for got, bound, base, other in ((dx, r.dx_bound, x, w), (dw, r.dw_bound, w, x)):
        h = torch.randn(base.shape, dtype=torch.float64, device=DEV) * 1e-4
        a, b = base.double(), other.double()
        both = (lambda t: L(t, b)) if base is x else (lambda t: L(b, t))
        want = (both(a + h) - both(a - h)) / 2
        # third differences of a log-sum-exp: at most |dz|^3 per token, with |dz| below 5e-3 here: 2e-7 of the weights' sum
        allowed = float((bound * h.abs()).sum()) + float(g.sum()) * (float(h.abs().amax()) * H ** 0.5 * 30) ** 3
        assert abs(float((got.double() * h).sum()) - want) <= allowed


def test_a_head_shared_by_two_losses():
    """Gradients of one weight from two batches add up in place."""
    torch.manual_seed(6)
    V, H = 300, 64
    xa, w, ya = inputs(50, H, V)
    xb, _, yb = inputs(90, H, V)
    dw = torch.zeros(V, H, device=DEV)
    want, bound, size = torch.zeros(V, H, dtype=torch.float64, device=DEV), 0, 0
    for x, y in ((xa, ya), (xb, yb)):
        g = torch.rand(len(y), device=DEV)
        _, lse = v4moe.linear_xent(x, w, y)
        v4moe.linear_xent_backward(x, w, y, lse, g, dw=dw, accumulate=True)
        r = Reference(x, w, y, g)
        want, bound, size = want + r.dw, bound + r.dw_bound, size + r.dw_size
    close(dw, want, bound + 2 * 2.0 ** -23 * size, "dw")


def test_graph_replays():
    torch.manual_seed(7)
    T, H, V = 90, 101, 700
    x, w, y = inputs(T, H, V)
    g = torch.rand(T, device=DEV)

    def step():
        loss, lse = v4moe.linear_xent(x, w, y)
        return loss, lse, *v4moe.linear_xent_backward(x, w, y, lse, g)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn_like(x))
        y.copy_(torch.randint(-30 * i, V, (T,), device=DEV))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams():
    torch.manual_seed(8)
    a, b = inputs(200, 256, 3000), inputs(100, 128, 5000)
    want = [v4moe.linear_xent(*v) for v in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, v in zip(streams, (a, b)):
        with torch.cuda.stream(s):
            got.append(v4moe.linear_xent(*v))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for u, v in zip(got, want) for p, q in zip(u, v))


def test_python_refusals():
    x, w, y = inputs(6, 16, 40)
    _, lse = v4moe.linear_xent(x, w, y)
    g = torch.ones(6, device=DEV)
    for bad in (dict(x=x.float()), dict(w=w.float()), dict(w=w[:, :8]), dict(targets=y.int()), dict(targets=y[:5]),
                dict(targets=y.cpu()), dict(x=x.cpu()), dict(w=w.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            v4moe.linear_xent(**{**dict(x=x, w=w, targets=y), **bad})
    for bad in (dict(lse=lse[:5]), dict(lse=lse.double()), dict(dloss=g[:5]), dict(dloss=g.to(BF16)), dict(dloss=g.cpu()),
                dict(accumulate=True), dict(dx=torch.empty(6, 15, device=DEV)), dict(dw=torch.empty(39, 16, device=DEV)),
                dict(dw=torch.empty(40, 16, dtype=torch.float16, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            v4moe.linear_xent_backward(**{**dict(x=x, w=w, targets=y, lse=lse, dloss=g), **bad})
