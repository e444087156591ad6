"""Every tile of the grouped products and of the cross entropy against sums in 64 bits.

Which tile a call takes is read from the library (a table of measured times decides), and each case says the one that
it is here for: if the table changes, the case fails before it stops covering its tile.

Bounds.  An element of a product is one chain of fp32 additions of exact bf16 products, in instructions of 32 terms: off
by at most (n + 32) 2^-23 of the sum of its n products' magnitudes, and rounded once, by half a step of its type.  The
cross entropy: a logit is off by ez, as such a sum; the log-sum-exp by el = ez + (range + 128 + V / 4096) 2^-22; d is off
by p (ez + el) and rounded to bf16 (2^-8), at the target by 2^-16."""
import itertools

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
FORWARD, DX, DW, AGAIN, SHARED = 0, 1, 2, 3, 1 << 30


def tile(code):
    return ("shared " if code & SHARED else "") + f"{(code & ~SHARED) >> 16}x{code & 0xFFFF}"


def grouped_tile(counts, N, K, what, both=0):
    return tile(v4moe.lib().moe_grouped_tile(sum(counts), len(counts), N, K, what, both))


def xent_tile(T, H, V, what, both=0):
    return tile(v4moe.lib().moe_linear_xent_tile(T, H, V, what, both))


def randn(*shape, std=1.0):
    return torch.randn(*shape, dtype=F32, device=DEV).mul_(std).to(BF16)


def rows(n, cols, pad=0, std=1.0):
    return randn(n, cols + pad, std=std)[:, :cols]


def offsets_of(counts):
    return torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32, device=DEV)


def close(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


# Rows of each expert (many with a last tile of few rows, one row, none), N, K, and the tiles of y, of dx alone, of dW
# alone and of both together
GROUPED = [
    ([5, 0, 1, 2], 264, 328, "16x64", "16x64", "64x64", "16x64", "64x64"),
    ([700, 0, 1, 300, 64], 264, 320, "32x64", "32x64", "64x64", "32x64", "64x64"),
    ([900, 0, 1200, 901], 520, 448, "64x64", "32x64", "64x64", "32x64", "64x64"),
    ([300, 20] * 16, 72, 72, "64x64", "64x64", "64x64", "shared 128x128", "shared 128x128"),
    ([300, 20] * 16, 520, 72, "128x128", "64x64", "64x64", "shared 128x128", "shared 128x128"),
    ([300, 20] * 16, 521, 73, "128x128", "64x64", "64x64", "shared 128x128", "shared 128x128"),
    ([300, 20] * 16, 72, 520, "64x64", "128x128", "64x64", "shared 128x128", "shared 128x128"),
    ([2000, 1, 0, 900], 4104, 72, "256x256", "32x64", "64x64", "32x64", "64x64"),
    ([2000, 1, 0, 900], 4099, 77, "256x256", "32x64", "64x64", "32x64", "64x64"),
    ([2000, 1, 0, 900], 72, 4104, "32x64", "256x256", "64x64", "256x256", "64x64"),
    ([2000, 1, 0, 900], 77, 4099, "32x64", "256x256", "64x64", "256x256", "64x64"),
    ([200, 0, 1, 130], 2056, 2056, "64x64", "64x64", "128x128", "64x64", "128x128"),
    ([40, 0, 1], 2056, 2056, "16x64", "16x64", "256x256", "16x64", "256x256"),
    ([330, 0, 1], 2051, 2059, "64x64", "64x64", "256x256", "64x64", "256x256"),
    ([6000, 1, 0, 2100], 72, 2056, "64x64", "128x128", "64x64", "128x128", "64x64"),
    ([1400, 0, 1, 1500], 4104, 1032, "256x256", "128x128", "128x128", "128x128", "128x128"),
    ([1400, 0, 1, 1500], 1032, 4104, "128x128", "256x256", "128x128", "256x256", "128x128"),
    ([700, 130, 1, 0, 400], 2056, 1032, "64x64", "32x64", "128x128", "32x64", "128x128"),
]


def test_every_tile_of_the_grouped_products_is_here():
    for counts, N, K, y, dx, dw, both_dx, both_dw in GROUPED:
        got = [grouped_tile(counts, N, K, *a) for a in ((FORWARD,), (DX,), (DW,), (DX, 1), (DW, 1))]
        assert got == [y, dx, dw, both_dx, both_dw], (counts, N, K, got)
    sizes = ["16x64", "32x64", "64x64", "128x128", "256x256"]
    assert {c[3] for c in GROUPED} == {c[4] for c in GROUPED} == set(sizes) and {c[5] for c in GROUPED} == set(sizes[2:])
    assert any(c[6].startswith("shared") for c in GROUPED)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_grouped(case, pad):
    counts, N, K = GROUPED[case][:3]
    torch.manual_seed(case)
    M, E, off = sum(counts), len(counts), offsets_of(counts)
    x, dy, w = rows(M, K, pad), rows(M, N, pad), randn(E, N, K)
    f = lambda *s: torch.zeros(*s, dtype=torch.float64, device=DEV)  # noqa: E731
    y, ys, dx, dxs, dw, dws = f(M, N), f(M, N), f(M, K), f(M, K), f(E, N, K), f(E, N, K)
    for e, (i, j) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        a, b, d = x[i:j].double(), w[e].double(), dy[i:j].double()
        y[i:j], ys[i:j] = a @ b.t(), a.abs() @ b.abs().t()
        dx[i:j], dxs[i:j] = d @ b, d.abs() @ b.abs()
        dw[e], dws[e] = d.t() @ a, d.abs().t() @ a.abs()
    most = max(counts)
    for t in (BF16, F32):
        new = lambda *s: torch.full(s, 7.0, dtype=t, device=DEV)  # noqa: E731
        out = new(M, N + pad)
        close(v4moe.grouped_linear(x, w, off, out=out[:, :N]), y, (K + 32) * 2.0 ** -23 * ys, "y")
        assert bool((out[:, N:] == 7.0).all())
        gx, gw = new(M, K + pad), new(E, N, K)
        v4moe.grouped_linear_backward(x, dy, w, off, dx=gx[:, :K], dw=gw)                        # both
        close(gx[:, :K], dx, (N + 32) * 2.0 ** -23 * dxs, "dx")
        close(gw, dw, (most + 32) * 2.0 ** -23 * dws, "dw")
        assert bool((gx[:, K:] == 7.0).all())
        assert torch.equal(v4moe.grouped_linear_backward(x, dy, w, off, dx=new(M, K), need_dw=False)[0], gx[:, :K])   # each alone
        assert torch.equal(v4moe.grouped_linear_backward(x, dy, w, off, dw=new(E, N, K), need_dx=False)[1], gw)
        before = torch.randn(E, N, K, dtype=F32, device=DEV).to(t)
        for alone in (False, True):
            after = before.clone()
            v4moe.grouped_linear_backward(x, dy, w, off, dw=after, accumulate=True, need_dx=not alone)
            close(after, before.double() + dw, (most + 33) * 2.0 ** -23 * (dws + before.double().abs()), "dw added to")
            for e, n in enumerate(counts):
                assert n or torch.equal(after[e], before[e])


@pytest.mark.gpu
@pytest.mark.parametrize("what", [FORWARD, DX])
def test_a_row_of_a_grouped_product_is_the_same_in_every_tile(what):
    """Every bit of y and of dx: batches of one expert whose rows are the first of a larger one's, in every tile."""
    torch.manual_seed(what)
    N, K, batches = 4104, 264, [3000, 2000, 700, 500, 300, 200, 100, 40, 5, 1]
    if what == DX:
        N, K = K, N
    tiles = {grouped_tile([m], N, K, what) for m in batches}
    assert tiles == {"16x64", "32x64", "64x64", "128x128", "256x256"}
    x, w = rows(3000, K if what == FORWARD else N), randn(1, N, K)

    def run(m, t):
        off, out = offsets_of([m]), torch.empty(m, N if what == FORWARD else K, dtype=t, device=DEV)
        if what == FORWARD:
            return v4moe.grouped_linear(x[:m], w, off, out=out)
        return v4moe.grouped_linear_backward(torch.zeros(m, K, dtype=BF16, device=DEV), x[:m], w, off, dx=out, need_dw=False)[0]

    for t in (BF16, F32):
        whole = run(batches[0], t)
        for m in batches[1:]:
            assert torch.equal(run(m, t), whole[:m]), m


@pytest.mark.gpu
def test_a_weights_gradient_is_the_same_in_every_tile():
    """Every bit of dW: an expert's part of it, alone and among others, with fewer columns and rows of dW, in every tile."""
    torch.manual_seed(3)
    M, N, K = 330, 2056, 2056
    x, dy, w = rows(M, K), rows(M, N), randn(3, N, K)
    _, whole = v4moe.grouped_linear_backward(x, dy, w, offsets_of([0, M, 0]), need_dx=False)
    tiles = {grouped_tile([0, M, 0], N, K, DW)}
    for n, k in ((2056, 1544), (2056, 1032), (520, 264), (136, 72)):
        _, part = v4moe.grouped_linear_backward(x[:, :k], dy[:, :n], w[1:2, :n, :k].contiguous(), offsets_of([M]), need_dx=False)
        tiles.add(grouped_tile([M], n, k, DW))
        assert torch.equal(part[0], whole[1, :n, :k])
    assert tiles == {"64x64", "128x128", "256x256"}


# T, H, V, and the tiles of the loss's logits, the gradients' logits, dx and dW in one call, dx alone
XENT = [
    (5, 64, 300, "16x256", "16x256", "shared 128x128", "shared 128x128", "32x64"),
    (17, 72, 1000, "32x256", "32x256", "shared 128x128", "shared 128x128", "32x64"),
    (40, 136, 1000, "64x256", "64x256", "shared 128x128", "shared 128x128", "32x64"),
    (100, 2049, 300, "128x128", "128x128", "shared 128x128", "shared 128x128", "64x64"),
    (1500, 264, 4099, "128x128", "128x128", "shared 128x128", "shared 128x128", "64x64"),
    (2000, 2056, 300, "128x128", "128x128", "shared 128x128", "shared 128x128", "128x128"),
    (2000, 2056, 4099, "128x128", "128x128", "shared 128x128", "shared 128x128", "256x256"),
    (1000, 1032, 33000, "128x128", "128x128", "128x128", "256x256", "128x128"),
    (1000, 2056, 33000, "128x128", "128x128", "256x256", "256x256", "256x256"),
    (1000, 505, 60003, "256x256", "256x256", "128x128", "256x256", "128x128"),
    (4100, 1025, 70001, "256x256", "256x256", "shared 128x128", "shared 128x128", "256x256"),          # in three pieces
    (4100, 2056, 70000, "256x256", "256x256", "256x256", "256x256", "256x256"),                         # the same
]


def test_every_tile_of_the_cross_entropy_is_here():
    for T, H, V, *want in XENT:
        got = [xent_tile(T, H, V, *a) for a in ((FORWARD,), (AGAIN,), (DX, 1), (DW, 1), (DX,))]
        assert got == want, (T, H, V, got)
    few, square = {"16x256", "32x256", "64x256"}, {"128x128", "256x256"}
    assert {c[3] for c in XENT} == {c[4] for c in XENT} == few | square
    assert {c[5] for c in XENT} == square | {"shared 128x128"} and {c[6] for c in XENT} == {"256x256", "shared 128x128"}
    assert {c[7] for c in XENT} == {"32x64", "64x64"} | square


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(XENT)))
@pytest.mark.parametrize("pad", [0, 3])
def test_xent(case, pad):
    T, H, V = XENT[case][:3]
    torch.manual_seed(case)
    x, w = rows(T, H, pad), rows(V, H, pad, 1.5 * H ** -0.5)
    y = torch.randint(0, V, (T,), device=DEV)
    y[torch.arange(T, device=DEV) % 4 == 1] = -100
    y[0], y[T // 2] = V - 1, V - 1
    g = (torch.rand(T, dtype=F32, device=DEV) + 0.1) / T
    k = torch.nonzero(y >= 0).flatten()
    n, at = len(k), torch.arange(len(k), device=DEV)
    a, b = x.double()[k], w.double()
    z = a @ b.t()
    ez = ((H + 32) * 2.0 ** -23 * (a.abs() @ b.abs().t())).amax(dim=1)
    exact = torch.logsumexp(z, dim=1)
    el = ez + (z.amax(dim=1) - z.amin(dim=1) + 128 + V / 4096) * 2.0 ** -22
    loss, lse = v4moe.linear_xent(x, w, y)
    close(lse[k], exact, el + exact.abs() * 2.0 ** -23, "lse")
    want = exact - z[at, y[k]]
    close(loss[k], want, ez + el + (exact.abs() + want.abs()) * 2.0 ** -23, "loss")
    none = y < 0
    assert not bool(loss[none].any()) and not bool(lse[none].any())

    d = torch.softmax(z, dim=1)
    del z
    gk = g.double()[k].unsqueeze(1)
    err = gk * d * (ez + el + exact.abs() * 2.0 ** -23 + 2.0 ** -22).unsqueeze(1) * 1.01
    d[at, y[k]] -= 1.0
    d *= gk
    target = d[at, y[k]].abs()
    err += d.abs() * (2.0 ** -8 + 2.0 ** -22)
    err[at, y[k]] -= target * (2.0 ** -8 - 2.0 ** -16)
    size = d.abs() + err
    f = lambda: torch.zeros(T, H, dtype=torch.float64, device=DEV)  # noqa: E731
    dx, dx_bound = f(), f()
    dx[k], dx_bound[k] = d @ b, err @ b.abs() + (V + 65) * 2.0 ** -23 * (size @ b.abs())
    dw, dws = d.t() @ a, size.t() @ a.abs()
    dw_bound = err.t() @ a.abs() + (2 * n + 64) * 2.0 ** -23 * dws
    del d, err, size
    for t in (BF16, F32):
        new = lambda *s: torch.full(s, 7.0, dtype=t, device=DEV)  # noqa: E731
        gx, gw = new(T, H + pad), new(V, H + pad)
        v4moe.linear_xent_backward(x, w, y, lse, g, dx=gx[:, :H], dw=gw[:, :H])
        close(gx[:, :H], dx, dx_bound, "dx")
        close(gw[:, :H], dw, dw_bound, "dw")
        assert bool((gx[:, H:] == 7.0).all()) and bool((gw[:, H:] == 7.0).all()) and not bool(gx[:, :H][none].any())
        close(v4moe.linear_xent_backward(x, w, y, lse, g, dx=new(T, H), need_dw=False)[0], dx, dx_bound, "dx alone")
        assert torch.equal(v4moe.linear_xent_backward(x, w, y, lse, g, dw=new(V, H), need_dx=False)[1], gw[:, :H])
        before = torch.randn(V, H, dtype=F32, device=DEV).mul_(1 / T).to(t)
        after = before.clone()
        v4moe.linear_xent_backward(x, w, y, lse, g, dw=after, accumulate=True)
        close(after, before.double() + dw, dw_bound + 2.0 ** -23 * (before.double().abs() + dws), "dw added to")


@pytest.mark.gpu
def test_a_token_is_the_same_in_every_tile():
    """Every bit of loss and log-sum-exp: batches whose tokens are the first of a larger one's, in every tile."""
    torch.manual_seed(5)
    H, V, batches = 264, 33000, [4100, 1000, 300, 65, 64, 33, 17, 16, 3, 1]
    assert {xent_tile(t, H, V, FORWARD) for t in batches} == {"16x256", "32x256", "64x256", "128x128", "256x256"}
    x, w, y = rows(4100, H), rows(V, H, 0, 1.5 * H ** -0.5), torch.randint(-V // 8, V, (4100,), device=DEV)
    loss, lse = v4moe.linear_xent(x, w, y)
    for t in batches[1:]:
        a, b = v4moe.linear_xent(x[:t], w, y[:t])
        assert torch.equal(a, loss[:t]) and torch.equal(b, lse[:t]), t


def test_refusals():
    for bad in ((-1, 3, 16, 32, 0, 0), (6, 0, 16, 32, 0, 0), (6, 3, 0, 32, 0, 0), (6, 3, 16, 0, 0, 0), (6, 3, 16, 32, 3, 0),
                (6, 3, 16, 32, -1, 0)):
        assert v4moe.lib().moe_grouped_tile(*bad) == 0
    for bad in ((0, 32, 100, 0, 0), (-1, 32, 100, 0, 0), (5, 0, 100, 0, 0), (5, 32, 0, 0, 0), (5, 32, 100, 4, 0), (5, 32, 100, -1, 0)):
        assert v4moe.lib().moe_linear_xent_tile(*bad) == 0
