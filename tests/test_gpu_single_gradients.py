"""Gradients asked for one at a time: what is not needed is neither computed nor allocated, and what is equals what a call
for all of them gives.

Bits: a gradient's sums are the same in a call of its own, but for the cross entropy's dx, whose slices of the
vocabulary are cut for its tile alone: it is compared with the formula in 64 bits (bounds as in the other tests of these
gradients: a logit's fp32 sum, d rounded to bf16, the products' sums)."""
import itertools

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


def subsets(names):
    return [s for k in range(1, len(names)) for s in itertools.combinations(names, k)]


def grown(call):
    """What a call returns, and the most memory that it had beyond what there was before."""
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    out = call()
    return out, torch.cuda.max_memory_allocated() - before


# a few rows and many; gradients that share a launch and that do not; operands that are copied first
@pytest.mark.parametrize("counts,N,K,pad", [([3, 0, 5], 64, 72, 0), ([300, 290], 257, 259, 3), ([900, 0, 1200, 901], 320, 448, 0),
                                            ([2000, 3000], 1024, 1024, 8)])
def test_grouped(counts, N, K, pad):
    torch.manual_seed(N)
    M, E = sum(counts), len(counts)
    x, dy, w = rows(M, K, pad), rows(M, N, pad), torch.randn(E, N, K, device=DEV).to(BF16)
    off = torch.tensor([0, *itertools.accumulate(counts)], dtype=torch.int32, device=DEV)
    dx, dw = v4moe.grouped_linear_backward(x, dy, w, off)
    a, none = v4moe.grouped_linear_backward(x, dy, w, off, need_dw=False)
    assert none is None and torch.equal(a, dx)
    none, b = v4moe.grouped_linear_backward(x, dy, w, off, need_dx=False)
    assert none is None and torch.equal(b, dw)
    # into given ones, added to
    held = torch.randn(E, N, K, device=DEV)
    both, one = held.clone(), held.clone()
    v4moe.grouped_linear_backward(x, dy, w, off, dw=both, accumulate=True)
    v4moe.grouped_linear_backward(x, dy, w, off, dw=one, accumulate=True, need_dx=False)
    assert torch.equal(both, one)
    given = torch.empty(M, K, device=DEV)
    v4moe.grouped_linear_backward(x, dy, w, off, dx=given, need_dw=False)
    assert torch.equal(given.to(BF16), dx)


def test_grouped_without_weights_gradient_takes_no_room_for_it():
    x, dy, w = rows(64, 256), rows(64, 512), torch.randn(16, 512, 256, device=DEV).to(BF16)
    off = torch.arange(0, 65, 4, dtype=torch.int32, device=DEV)
    _, most = grown(lambda: v4moe.grouped_linear_backward(x, dy, w, off, need_dw=False))
    assert most < w.numel() * 2
    _, most = grown(lambda: v4moe.grouped_linear_backward(x, dy, w, off))
    assert most >= w.numel() * 2


class Loss:
    """Gradients of the cross entropy in 64 bits with their bounds."""

    def __init__(self, x, w, y, g):
        T, (V, H) = x.shape[0], w.shape
        k = torch.nonzero((y >= 0) & (y < V)).flatten()
        a, b, n = x.double()[k], w.double(), len(k)
        z = a @ b.t()
        ez = ((H + 32) * 2.0 ** -23 * (a.abs() @ b.abs().t())).amax(dim=1)
        lse = torch.logsumexp(z, dim=1)
        el = ez + (z.amax(dim=1) - z.amin(dim=1) + 128 + V / 4096) * 2.0 ** -22 + lse.abs() * 2.0 ** -23
        p = torch.softmax(z, dim=1)
        gk = g.double()[k].unsqueeze(1)
        err = gk.abs() * p * (ez + el + 2.0 ** -22).unsqueeze(1) * 1.01
        d = p.clone()
        d[torch.arange(n, device=DEV), y[k]] -= 1.0
        d *= gk
        err += d.abs() * (2.0 ** -8 + 2.0 ** -22)
        size = d.abs() + err
        self.dx, self.dx_bound = (torch.zeros(T, H, dtype=torch.float64, device=DEV) for _ in range(2))
        self.dx[k], self.dx_bound[k] = d @ b, err @ b.abs() + (V + 65) * 2.0 ** -23 * (size @ b.abs())


# few tokens and many: every tile of dx alone, with its slices of the vocabulary
@pytest.mark.parametrize("T,H,V,pad", [(1, 64, 300, 0), (20, 512, 9000, 0), (60, 1001, 5000, 3), (300, 256, 20000, 0), (300, 2048, 4099, 8),
                                       (2000, 512, 9001, 0), (3000, 2048, 4096, 0), (4100, 32, 66000, 0)])
def test_xent(T, H, V, pad):
    torch.manual_seed(T + V)
    x, w = rows(T, H, pad), rows(V, H, pad, 1.5 * H ** -0.5)
    y = torch.randint(-V // 4, V, (T,), device=DEV)
    y[0] = V - 1
    g = (torch.rand(T, device=DEV) + 0.1) / T
    _, lse = v4moe.linear_xent(x, w, y)
    r = Loss(x, w, y, g)
    for t in (BF16, F32):
        dx, none = v4moe.linear_xent_backward(x, w, y, lse, g, dx=torch.empty(T, H, dtype=t, device=DEV), need_dw=False)
        assert none is None
        half = torch.finfo(t).eps / 2
        bad = ~((dx.double() - r.dx).abs() <= r.dx_bound * (1 + half) + half * r.dx.abs())
        assert not bool(bad.any()), (int(bad.sum()), float((dx.double() - r.dx).abs().max()))
        again, _ = v4moe.linear_xent_backward(x, w, y, lse, g, dx=torch.empty(T, H, dtype=t, device=DEV), need_dw=False)
        assert torch.equal(dx, again)
    _, dw = v4moe.linear_xent_backward(x, w, y, lse, g)
    none, alone = v4moe.linear_xent_backward(x, w, y, lse, g, need_dx=False)
    assert none is None and torch.equal(alone, dw)


def test_xent_of_a_frozen_head_takes_no_room_for_its_gradient():
    x, w = rows(16, 512), rows(40000, 512, std=0.05)
    y, g = torch.arange(16, device=DEV), torch.ones(16, device=DEV)
    _, lse = v4moe.linear_xent(x, w, y)
    _, most = grown(lambda: v4moe.linear_xent_backward(x, w, y, lse, g, need_dw=False))
    assert most < w.numel() * 2


# unlisted rows and listed ones, several of the ranks' pieces, one launch for the gradients and two
@pytest.mark.parametrize("M,N,K,r,L,pad", [(9, 64, 72, 4, 3, 0), (50, 128, 136, 100, 2, 3), (700, 256, 320, 16, 5, 0), (700, 65, 77, 40, 5, 3),
                                           (3000, 264, 328, 64, 4, 0), (3000, 264, 328, 100, 4, 0), (1500, 128, 128, 8, 1500, 0)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_lora(M, N, K, r, L, pad, accumulate):
    torch.manual_seed(M + r)
    q = dict(x=rows(M, K, pad), dy=rows(M, N, pad), a=torch.randn(L, r, K, device=DEV).to(BF16),
             b=torch.randn(L, r, N, device=DEV).to(BF16), ids=torch.randint(-1, L, (M,), device=DEV).to(torch.int32),
             scale=torch.rand(L, device=DEV))
    base = rows(M, K)
    held = dict(da=torch.randn(L, r, K, device=DEV), db=torch.randn(L, r, N, device=DEV))

    def call(names):
        given = {n: held[n].clone() for n in ("da", "db") if n in names} if accumulate else {}
        more = dict(base=base) if "dx" in names else {}
        out = v4moe.lora_backward(**q, **more, **given, accumulate=bool(given), **{"need_" + n: n in names for n in ("dx", "da", "db")})
        return dict(zip(("dx", "da", "db"), out))

    want = call(("dx", "da", "db"))
    for names in subsets(("dx", "da", "db")):
        got = call(names)
        for n in want:
            assert got[n] is None if n not in names else torch.equal(got[n], want[n]), (names, n)


def test_refusals():
    x, dy, w = rows(8, 16), rows(8, 24), torch.randn(2, 24, 16, device=DEV).to(BF16)
    off = torch.tensor([0, 5, 8], dtype=torch.int32, device=DEV)
    q = dict(x=x, dy=dy, w=w, offsets=off)
    for bad in (dict(need_dx=False, need_dw=False), dict(need_dx=False, dx=torch.empty(8, 16, device=DEV)),
                dict(need_dw=False, dw=torch.empty_like(w)), dict(need_dw=False, accumulate=True)):
        with pytest.raises(ValueError):
            v4moe.grouped_linear_backward(**q, **bad)
    head, y, f = rows(30, 16), torch.zeros(8, dtype=torch.int64, device=DEV), torch.ones(8, device=DEV)
    q = dict(x=x, w=head, targets=y, lse=f, dloss=f)
    for bad in (dict(need_dx=False, need_dw=False), dict(need_dx=False, dx=torch.empty(8, 16, device=DEV)),
                dict(need_dw=False, dw=torch.empty_like(head)), dict(need_dw=False, accumulate=True)):
        with pytest.raises(ValueError):
            v4moe.linear_xent_backward(**q, **bad)
    a, b = torch.randn(2, 3, 16, device=DEV).to(BF16), torch.randn(2, 3, 24, device=DEV).to(BF16)
    q = dict(x=x, dy=dy, a=a, b=b, ids=torch.zeros(8, dtype=torch.int32, device=DEV), scale=f[:2])
    none = dict(need_dx=False, need_da=False, need_db=False)
    for bad in (none, dict(need_dx=False, base=x), dict(need_dx=False, dx=torch.empty_like(x)), dict(need_da=False, da=torch.empty_like(a)),
                dict(need_db=False, db=torch.empty_like(b)), dict(accumulate=True, need_da=False, need_db=False),
                dict(accumulate=True, need_da=False), dict(accumulate=True, da=torch.empty_like(a))):
        with pytest.raises(ValueError):
            v4moe.lora_backward(**{**q, **bad})
