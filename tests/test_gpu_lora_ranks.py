"""Adapters of ranks above 64, whose factors pass in pieces of 64 ranks, on rows listed by adapter and on few rows as they
come, against the formulas in 64 bits.

Bounds: u = scale A x is off by (K + 64) 2^-23 of the sum of its products' magnitudes and kept to 2^-16; what is made of it
is a sum of twice r (or twice the rows') products, added to the base, and rounded once by half a step."""
import ctypes

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
STEP32 = 2.0 ** -23

# rows, columns, inputs, rank, adapters, whether the forward and the gradients have their rows listed
CASES = [
    (3000, 264, 328, 65, 5, True, True), (3000, 257, 321, 100, 5, True, True), (2500, 128, 136, 128, 4, True, True),
    (1100, 520, 264, 256, 16, True, True), (1500, 72, 1032, 512, 7, True, True), (130, 65, 77, 129, 9, False, True),
    (60, 264, 328, 192, 5, False, False), (17, 7, 9, 512, 3, False, False), (3000, 72, 64, 80, 40, True, True),
]


def test_listed_as_said():
    """(The workspace holds the list beside u, and in a backward du.)"""
    for M, N, K, r, L, forward, backward in CASES:
        p = v4moe.LoraC(M, N, K, r, L)
        u = (M * 2 * ((r + 15) // 16 * 16) * 2 + 255) // 256 * 256
        need = [v4moe.lib().moe_lora_workspace_bytes(ctypes.byref(p), k) for k in (0, 1)]
        assert [need[0] > u, need[1] > 2 * u] == [forward, backward], (M, r, L)


def rows(n, cols, pad, t=BF16):
    return torch.randn(n, cols + pad, dtype=F32, device=DEV).to(t)[:, :cols]


def close(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


class Formula:
    """One product pair in 64 bits: u = scale F v of each row, and what is made of it."""

    def __init__(self, v, f, ids, scale):
        self.ids, (self.L, r, K) = ids, f.shape
        self.u, self.err = (torch.zeros(v.shape[0], r, dtype=torch.float64, device=DEV) for _ in range(2))
        for i in range(self.L):
            k = ids == i
            p, q, s = v[k].double(), f[i].double(), scale[i].double()
            self.u[k] = s * (p @ q.t())
            self.err[k] = s * ((K + 64) * STEP32 * (p.abs() @ q.abs().t())) + self.u[k].abs() * (2.0 ** -16 + 2.0 ** -22)

    def expanded(self, f, base):
        out, bound, r = base.double().clone(), torch.zeros_like(base, dtype=torch.float64), f.shape[1]
        for i in range(self.L):
            k, q = self.ids == i, f[i].double()
            out[k] += self.u[k] @ q
            bound[k] = self.err[k] @ q.abs() + (2 * r + 64) * STEP32 * ((self.u[k].abs() + self.err[k]) @ q.abs()) + STEP32 * out[k].abs()
        return out, bound

    def summed(self, v):
        d, bound = (torch.zeros(self.L, self.u.shape[1], v.shape[1], dtype=torch.float64, device=DEV) for _ in range(2))
        for i in range(self.L):
            k = self.ids == i
            p, e, q = self.u[k], self.err[k], v[k].double()
            d[i] = p.t() @ q
            bound[i] = e.t() @ q.abs() + (2 * int(k.sum()) + 128) * STEP32 * ((p.abs() + e).t() @ q.abs())
        return d, bound


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("t", [BF16, F32])
def test_result_and_gradients(case, pad, t):
    M, N, K, r, L = CASES[case][:5]
    torch.manual_seed(case)
    a, b = (torch.randn(L, r, n, dtype=F32, device=DEV).mul_(s ** -0.5).to(BF16) for n, s in ((K, K), (N, r)))
    x, dy, y, base = rows(M, K, pad), rows(M, N, pad), rows(M, N, pad, t), rows(M, K, pad, t)
    ids = torch.randint(-1, L, (M,), device=DEV).to(torch.int32)
    ids[ids == 1] = 0                                        # an adapter without rows
    scale = torch.rand(L, dtype=F32, device=DEV) + 0.5
    q = dict(x=x, a=a, b=b, ids=ids, scale=scale)
    none = ids < 0
    up, down = Formula(x, a, ids, scale), Formula(dy, b, ids, scale)
    out = v4moe.lora_add(y, **q)
    close(out, *up.expanded(b, y), "out")
    assert torch.equal(out[none], y[none])
    held = y.clone()
    assert torch.equal(v4moe.lora_add(held, **q, out=held), out)                       # in place
    new = lambda *s: torch.full(s, 7.0, dtype=t, device=DEV)  # noqa: E731
    dx, da, db = v4moe.lora_backward(dy=dy, base=base, **q, da=new(L, r, K), db=new(L, r, N))
    close(dx, *down.expanded(a, base), "dx")
    assert torch.equal(dx[none], base[none])
    (da_want, da_bound), (db_want, db_bound) = down.summed(x), up.summed(dy)
    close(da, da_want, da_bound, "da")
    close(db, db_want, db_bound, "db")
    if L > 1:
        assert not bool(da[1].any()) and not bool(db[1].any())
    pa, pb = torch.randn(L, r, K, dtype=F32, device=DEV).to(t), torch.randn(L, r, N, dtype=F32, device=DEV).to(t)
    ca, cb, mine = pa.clone(), pb.clone(), base.clone()
    v4moe.lora_backward(dy=dy, base=mine, dx=mine, **q, da=ca, db=cb, accumulate=True)
    assert torch.equal(mine, dx)
    close(ca, pa.double() + da_want, da_bound + STEP32 * (pa.double().abs() + da_want.abs()), "da added to")
    close(cb, pb.double() + db_want, db_bound + STEP32 * (pb.double().abs() + db_want.abs()), "db added to")
    # each gradient alone, and a row alone: the same bits
    assert torch.equal(v4moe.lora_backward(dy=dy, base=base, **q, need_da=False, need_db=False)[0], dx)
    assert torch.equal(v4moe.lora_backward(dy=dy, **q, da=new(L, r, K), need_dx=False, need_db=False)[1], da)
    assert torch.equal(v4moe.lora_backward(dy=dy, **q, db=new(L, r, N), need_dx=False, need_da=False)[2], db)
    some = torch.arange(0, M, max(M // 7, 1), device=DEV)
    few = dict(q, x=x[some].contiguous(), ids=ids[some].contiguous())
    assert torch.equal(v4moe.lora_add(y[some].contiguous(), **few), out[some])
    alone = v4moe.lora_backward(dy=dy[some].contiguous(), base=base[some].contiguous(), **few, need_da=False, need_db=False)[0]
    assert torch.equal(alone, dx[some])
