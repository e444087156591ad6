"""Products grouped by expert against sums in 64 bits.

Bounds: an element is one chain of fp32 additions of exact bf16 products, in matrix
instructions of 32 terms: off by at most (n + 32) 2^-23 of the sum of its n products'
magnitudes (an addition is off by 2^-24 of its result, twice that allows the
instruction's inner sums to be cut off instead of rounded), and rounded once: by 2^-8 of
the value where it is bf16, 2^-24 where it is fp32."""
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


def close(got, want, size, n, what, rounding=1):
    half = torch.finfo(got.dtype).eps / 2
    bound = half * rounding * want.abs() + (n + 32) * 2.0 ** -23 * (1 + half) * size
    bad = (got.double() - want).abs() > bound
    assert not bool(bad.any()) and not bool(got.isnan().any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


def rows(n, cols, pad=0, at=0, std=1.0):
    """bf16 rows [n][cols] inside wider ones, `at` elements into the buffer."""
    buf = torch.randn(n * (cols + pad) + at, device=DEV).mul_(std).to(BF16)
    return buf[at:].view(n, cols + pad)[:, :cols]


def offsets_of(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device=DEV)


def reference(x, w, off, dy=None):
    """y, and with dy (dx, dw), with the sums of the products' magnitudes of each, in 64 bits."""
    at = off.tolist()
    M, (E, N, K) = x.shape[0], w.shape
    f = lambda *s: torch.zeros(*s, dtype=torch.float64, device=DEV)  # noqa: E731
    y, ys, dx, dxs, dw, dws = f(M, N), f(M, N), f(M, K), f(M, K), f(E, N, K), f(E, N, K)
    for e in range(E):
        s = slice(at[e], at[e + 1])
        a, b = x[s].double(), w[e].double()
        y[s], ys[s] = a @ b.t(), a.abs() @ b.abs().t()
        if dy is not None:
            d = dy[s].double()
            dx[s], dxs[s] = d @ b, d.abs() @ b.abs()
            dw[e], dws[e] = d.t() @ a, d.abs().t() @ a.abs()
    return (y, ys), (dx, dxs), (dw, dws)


# rows of each expert, N, K: every tile (by the mean rows), experts without rows, one row, tiles that end at, before and
# after an expert's rows; contractions of one step, of less, of many, of a partial last one; sizes that no tile divides
SHAPES = [
    ([1], 8, 8), ([0, 1, 0], 16, 32), ([3, 0, 5, 1], 64, 64), ([0, 0, 0, 0], 64, 64), ([16, 15, 17, 1, 0, 2], 72, 136),
    ([33, 1, 20, 40], 200, 264), ([65, 0, 63, 64, 1], 128, 192), ([129, 64, 130, 1], 264, 320), ([128, 127], 136, 64),
    ([257, 255, 256, 0, 300], 520, 448), ([700], 256, 512), ([1] * 40 + [0] * 24, 128, 128), ([5, 200, 0, 90], 33, 47),
    ([300, 290], 257, 259), ([2, 3], 1, 1), ([40], 7, 4096), ([520], 1032, 72),
]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("pad", [0, 8, 5])
def test_products_and_gradients(counts, N, K, pad):
    torch.manual_seed(sum(counts) + N + K + pad)
    M, E = sum(counts), len(counts)
    x, dy = rows(M, K, pad), rows(M, N, pad)
    w = torch.randn(E, N, K, device=DEV).to(BF16)
    off = offsets_of(counts)
    (y, ys), (dx, dxs), (dw, dws) = reference(x, w, off, dy)
    for t in (BF16, F32):
        out = torch.full((M, N + pad), 7.0, dtype=t, device=DEV)
        got = v4moe.grouped_linear(x, w, off, out=out[:, :N])
        close(got, y, ys, K, "y")
        assert bool((out[:, N:] == 7.0).all())
        gx = torch.full((M, K + pad), 7.0, dtype=t, device=DEV)
        gw = torch.full((E, N, K), 7.0, dtype=t, device=DEV)
        v4moe.grouped_linear_backward(x, dy, w, off, dx=gx[:, :K], dw=gw)
        close(gx[:, :K], dx, dxs, N, "dx")
        assert bool((gx[:, K:] == 7.0).all())
        longest = max(counts)
        close(gw, dw, dws, longest, "dw")
        before = torch.randn(E, N, K, device=DEV).to(t)
        sum_ = before.clone()
        v4moe.grouped_linear_backward(x, dy, w, off, dw=sum_, accumulate=True)
        close(sum_, before.double() + dw, before.double().abs() + dws, longest + 1, "dw added to")
        for e, n in enumerate(counts):
            assert n or torch.equal(sum_[e], before[e])


def test_default_types_and_determinism():
    torch.manual_seed(0)
    counts = [100, 0, 37, 260]
    x, dy, w, off = rows(397, 320), rows(397, 192), torch.randn(4, 192, 320, device=DEV).to(BF16), offsets_of(counts)
    y = v4moe.grouped_linear(x, w, off)
    dx, dw = v4moe.grouped_linear_backward(x, dy, w, off)
    assert y.dtype == dx.dtype == dw.dtype == BF16
    for _ in range(5):
        assert torch.equal(v4moe.grouped_linear(x, w, off), y)
        a, b = v4moe.grouped_linear_backward(x, dy, w, off)
        assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("count", [1, 20, 50, 100, 300])
def test_a_row_does_not_depend_on_the_others(count):
    """Every bit, whichever tile the batch has (the mean rows choose it)."""
    torch.manual_seed(count)
    N, K = 320, 1000
    x, dy, w = rows(700, K), rows(700, N), torch.randn(1, N, K, device=DEV).to(BF16)
    whole = offsets_of([700])
    y = v4moe.grouped_linear(x, w, whole, out=torch.empty(700, N, device=DEV))
    dx, _ = v4moe.grouped_linear_backward(x, dy, w, whole, dx=torch.empty(700, K, device=DEV))
    some = offsets_of([count])
    a = v4moe.grouped_linear(x[:count], w, some, out=torch.empty(count, N, device=DEV))
    b, _ = v4moe.grouped_linear_backward(x[:count], dy[:count], w, some, dx=torch.empty(count, K, device=DEV))
    assert torch.equal(a, y[:count]) and torch.equal(b, dx[:count])


def test_rows_of_no_expert_are_left_as_they_were():
    """... and what they hold reaches no gradient; neither do the rows of the next expert."""
    torch.manual_seed(1)
    counts, first, M, N, K = [30, 0, 70], 9, 140, 96, 128
    x, dy, w, off = rows(M, K), rows(M, N), torch.randn(3, N, K, device=DEV).to(BF16), offsets_of(counts, first)
    out_of = torch.ones(M, dtype=torch.bool, device=DEV)
    out_of[first:first + 100] = False
    clean = reference(x, w, off, dy)
    x[out_of], dy[out_of] = math.nan, math.inf
    y = v4moe.grouped_linear(x, w, off, out=torch.full((M, N), 5.0, device=DEV))
    dx, dw = v4moe.grouped_linear_backward(x, dy, w, off, dx=torch.full((M, K), 5.0, device=DEV),
                                           dw=torch.empty(3, N, K, device=DEV))
    assert bool((y[out_of] == 5.0).all()) and bool((dx[out_of] == 5.0).all())
    for got, (want, size), n in ((y, clean[0], K), (dx, clean[1], N), (dw, clean[2], 70)):
        if got.shape[0] == M:
            got, want, size = got[~out_of], want[~out_of], size[~out_of]
        close(got, want, size, n, "rows")
    # a NaN of one expert stays in its rows and its gradient
    x[first + 30:first + 100] = math.nan
    y = v4moe.grouped_linear(x, w, off)
    _, dw = v4moe.grouped_linear_backward(x, dy, w, off)
    assert not bool(y[first:first + 30].isnan().any()) and bool(y[first + 30:first + 100].isnan().all())
    assert not bool(dw[:2].isnan().any()) and bool(dw[2].isnan().all())


@pytest.mark.parametrize("at", [1, 4, 8])
def test_operands_that_begin_inside_a_buffer(at):
    torch.manual_seed(at)
    counts, N, K = [50, 20], 64, 72
    x, dy = rows(70, K, 8, at), rows(70, N, 8, at)
    w = torch.randn(2 * N * K + at, device=DEV).to(BF16)[at:].view(2, N, K)
    off = offsets_of(counts)
    (y, ys), (dx, dxs), (dw, dws) = reference(x, w, off, dy)
    buf = torch.empty(70 * N + at, dtype=BF16, device=DEV)
    close(v4moe.grouped_linear(x, w, off, out=buf[at:].view(70, N)), y, ys, K, "y")
    a, b = v4moe.grouped_linear_backward(x, dy, w, off)
    close(a, dx, dxs, N, "dx")
    close(b, dw, dws, 50, "dw")


def test_gradients_against_differences():
    """<dy, y(x + h) - y(x)> = <dx, h>, and so for the weights."""
    torch.manual_seed(2)
    counts, N, K = [9, 30, 0, 12], 48, 56
    x, dy = rows(51, K), rows(51, N)
    w, off = torch.randn(4, N, K, device=DEV).to(BF16), offsets_of(counts)
    dx, dw = v4moe.grouped_linear_backward(x, dy, w, off, dx=torch.empty(51, K, device=DEV), dw=torch.empty(4, N, K, device=DEV))
    y = lambda a, b: v4moe.grouped_linear(a, b, off, out=torch.empty(51, N, device=DEV)).double()  # noqa: E731
    hx = torch.randint(-1, 2, x.shape, device=DEV).to(BF16)
    hw = torch.randint(-1, 2, w.shape, device=DEV).to(BF16)
    # y is linear in each, so a difference over a whole step is y at the step; S: the magnitudes of all products
    for got, a, b in (((dx.double() * hx.double()).sum(), hx, w), ((dw.double() * hw.double()).sum(), x, hw)):
        want = (dy.double() * y(a, b)).sum()
        S = float((dy.double().abs() * reference(a, b, off)[0][1]).sum())
        assert abs(float(got - want)) <= (51 + N + K + 64) * 2.0 ** -23 * S


@pytest.mark.parametrize("bad", [[0, 50, 20, 64], [-5, 10, 900, 64], [64, 0, 64, 0], [2 ** 31 - 1, -2 ** 31, 7, 3], [0, 64, 0, 64]])
def test_offsets_that_do_not_ascend_touch_nothing_else(bad):
    """Results are unspecified, but what is written lies inside the outputs, and inputs are read inside theirs."""
    torch.manual_seed(3)
    guard = torch.full((96, 64), 3.0, device=DEV)
    x, dy, w = rows(64, 64), rows(64, 64), torch.randn(3, 64, 64, device=DEV).to(BF16)
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    v4moe.grouped_linear(x, w, off, out=guard[16:80])
    v4moe.grouped_linear_backward(x, dy, w, off, dx=guard[16:80])
    torch.cuda.synchronize()
    assert bool((guard[:16] == 3.0).all()) and bool((guard[80:] == 3.0).all())


def test_graph_replays():
    torch.manual_seed(4)
    counts, N, K = [70, 0, 50], 96, 101                      # (copies of the operands are captured too)
    x, dy, w, off = rows(120, K), rows(120, N), torch.randn(3, N, K, device=DEV).to(BF16), offsets_of(counts)
    v4moe.grouped_linear_backward(x, dy, w, off)
    y0 = v4moe.grouped_linear(x, w, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = v4moe.grouped_linear(x, w, off)
        dx, dw = v4moe.grouped_linear_backward(x, dy, w, off)
    for i in range(4):
        x.copy_(torch.randn_like(x))
        off.copy_(offsets_of([70 - 10 * i, 20 * i, 50 - 10 * i]))
        want = v4moe.grouped_linear(x, w, off), *v4moe.grouped_linear_backward(x, dy, w, off)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want))
    assert y0.shape == y.shape


def test_another_stream():
    torch.manual_seed(5)
    x, w, off = rows(300, 512), torch.randn(2, 256, 512, device=DEV).to(BF16), offsets_of([100, 200])
    want = v4moe.grouped_linear(x, w, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = v4moe.grouped_linear(x, w, off)
    s.synchronize()
    assert torch.equal(got, want)


def test_python_refusals():
    x, w, off = rows(8, 16), torch.randn(2, 24, 16, device=DEV).to(BF16), offsets_of([5, 3])
    dy = rows(8, 24)
    for bad in (dict(x=x.float()), dict(x=x[:, :8]), dict(w=w.float()), dict(w=w.transpose(1, 2)), dict(offsets=off.long()),
                dict(offsets=off[:2]), dict(offsets=off.cpu()), dict(x=x.cpu()), dict(out=torch.empty(8, 23, device=DEV)),
                dict(out=torch.empty(7, 24, device=DEV)), dict(x=x.t().contiguous().t())):
        with pytest.raises((ValueError, TypeError)):
            v4moe.grouped_linear(**{**dict(x=x, w=w, offsets=off), **bad})
    with pytest.raises(TypeError):
        v4moe.grouped_linear(x, w, off, out=torch.empty(8, 24, dtype=torch.float16, device=DEV))
    for bad in (dict(dy=dy[:, :8]), dict(dy=dy.float()), dict(accumulate=True), dict(dw=torch.empty(2, 16, 24, device=DEV)),
                dict(dx=torch.empty(8, 15, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            v4moe.grouped_linear_backward(**{**dict(x=x, dy=dy, w=w, offsets=off), **bad})
