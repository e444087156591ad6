"""Low-rank adapters of many requests against the formulas in 64 bits.

Bounds.  u = scale A x is summed in fp32 over slices of chains of matrix instructions: off
by at most (K + 64) 2^-23 of the sum of its products' magnitudes (twice an addition's
rounding, as the instructions may cut), scaled (2^-24), and kept as two bf16 numbers: 2^-8
of what the first left, 2^-16 of it.  What is made of it is a sum of r or of the rows'
products (twice as many, the two numbers' each), added to the base, and rounded once."""
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


def rows(n, cols, pad=0, t=BF16, at=0):
    buf = torch.randn(n * (cols + pad) + at, device=DEV).to(t)
    return buf[at:].view(n, cols + pad)[:, :cols]


def inputs(M, N, K, r, L, ids, pad=0):
    a, b = torch.randn(L, r, K, device=DEV).mul_(K ** -0.5).to(BF16), torch.randn(L, r, N, device=DEV).mul_(r ** -0.5).to(BF16)
    if ids == "runs":
        i = torch.randint(-1, L, (M // 30 + 2,), device=DEV)[torch.cumsum((torch.rand(M, device=DEV) < 0.03).int(), 0).clamp(max=M // 30 + 1)]
    elif ids == "any":
        i = torch.randint(-1, L, (M,), device=DEV)
    else:
        i = torch.full((M,), ids, device=DEV)
    return dict(x=rows(M, K, pad), a=a, b=b, ids=i.to(torch.int32), scale=torch.rand(L, device=DEV) + 0.5)


def factor(v, f, ids, scale):
    """scale[i] F[i] v[m] for every row, in 64 bits, 0 without an adapter; and its bound."""
    M, (L, r, K) = v.shape[0], f.shape
    u, bound = (torch.zeros(M, r, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(L):
        k = torch.nonzero(ids == i).flatten()
        if len(k):
            s, p, q = scale[i].double(), v.double()[k], f[i].double()
            u[k] = s * (p @ q.t())
            bound[k] = s.abs() * ((K + 64) * 2.0 ** -23 * (p.abs() @ q.abs().t())) + u[k].abs() * (2.0 ** -16 + 2.0 ** -22)
    return u, bound


def expanded(u, bound, f, ids, base):
    out, ob = base.double().clone(), torch.zeros_like(base, dtype=torch.float64)
    r = f.shape[1]
    for i in range(f.shape[0]):
        k = torch.nonzero(ids == i).flatten()
        if len(k):
            q = f[i].double()
            out[k] += u[k] @ q
            ob[k] = bound[k] @ q.abs() + (2 * r + 64) * 2.0 ** -23 * ((u[k].abs() + bound[k]) @ q.abs()) + 2.0 ** -23 * out[k].abs()
    return out, ob


def summed(u, bound, v, ids, L):
    d, db = (torch.zeros(L, u.shape[1], v.shape[1], dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(L):
        k = torch.nonzero(ids == i).flatten()
        p, q, e = u[k], v.double()[k], bound[k]
        if len(k):
            d[i] = p.t() @ q
            db[i] = e.t() @ q.abs() + (2 * len(k) + 128) * 2.0 ** -23 * ((p.abs() + e).t() @ q.abs())
    return d, db


def close(got, want, bound, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()))


# M, N, K, r, L, ids: one row; every tile and rank chunk; ranks of less than 16, of a partial 16, of more than 64; sizes
# that no tile divides, contractions of less than a slice and of a partial last one; each row another adapter, runs, one
# adapter, none; more rows than a list of the sums holds
CASES = [
    (1, 64, 64, 16, 1, 0), (1, 8, 8, 1, 3, "any"), (3, 7, 5, 3, 2, "any"), (16, 64, 256, 8, 20, "any"),
    (17, 72, 264, 16, 4, "any"), (64, 300, 520, 16, 64, "any"), (64, 256, 512, 64, 64, "any"), (100, 65, 1000, 24, 5, "runs"),
    (200, 129, 77, 33, 7, "any"), (300, 1001, 499, 64, 3, "runs"), (50, 128, 128, 100, 2, "any"), (40, 64, 700, 512, 2, "any"),
    (700, 256, 320, 16, 1, 0), (2300, 128, 256, 4, 9, "any"), (5000, 64, 136, 32, 6, "runs"), (2100, 200, 72, 64, 40, "any"),
    (30, 64, 64, 16, 4, -1), (30, 64, 64, 16, 4, 4), (9, 64, 4100, 16, 2, "any"),
]


@pytest.mark.parametrize("M,N,K,r,L,ids", CASES)
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("t", [BF16, F32])
def test_result_and_gradients(M, N, K, r, L, ids, pad, t):
    torch.manual_seed(M + N + K + r)
    q = inputs(M, N, K, r, L, ids, pad)
    y, dy, base = rows(M, N, pad, t), rows(M, N, pad), rows(M, K, pad, t)
    u, ub = factor(q["x"], q["a"], q["ids"], q["scale"])
    want, bound = expanded(u, ub, q["b"], q["ids"], y)
    none = (q["ids"] < 0) | (q["ids"] >= L)
    out = v4moe.lora_add(y, **q)
    assert out.dtype == t
    close(out, want, bound, "out")
    assert torch.equal(out[none], y[none])
    wide = torch.full((M, N + pad), 7.0, dtype=t, device=DEV)
    assert torch.equal(v4moe.lora_add(y, **q, out=wide[:, :N]), out) and bool((wide[:, N:] == 7.0).all())
    again = y.clone()
    assert torch.equal(v4moe.lora_add(again, **q, out=again), out)            # in place
    d, e = factor(dy, q["b"], q["ids"], q["scale"])
    dx_want, dx_bound = expanded(d, e, q["a"], q["ids"], base)
    da_want, da_bound = summed(d, e, q["x"], q["ids"], L)
    db_want, db_bound = summed(u, ub, dy, q["ids"], L)
    dx, da, db = v4moe.lora_backward(dy=dy, base=base, **q, da=torch.empty(L, r, K, dtype=t, device=DEV),
                                     db=torch.empty(L, r, N, dtype=t, device=DEV))
    assert dx.dtype == t
    close(dx, dx_want, dx_bound, "dx")
    assert torch.equal(dx[none], base[none])
    close(da, da_want, da_bound, "da")
    close(db, db_want, db_bound, "db")
    mine = base.clone()
    pa, pb = (torch.randn(*s.shape, device=DEV).to(t) for s in (da, db))
    ca, cb = pa.clone(), pb.clone()
    v4moe.lora_backward(dy=dy, base=mine, dx=mine, **q, da=ca, db=cb, accumulate=True)
    assert torch.equal(mine, dx)
    close(ca, pa.double() + da_want, da_bound + 2.0 ** -23 * (pa.double().abs() + da_want.abs()), "da added to")
    close(cb, pb.double() + db_want, db_bound + 2.0 ** -23 * (pb.double().abs() + db_want.abs()), "db added to")
    unused = torch.tensor([not bool((q["ids"] == i).any()) for i in range(L)], device=DEV)
    assert torch.equal(ca[unused], pa[unused]) and torch.equal(cb[unused], pb[unused])
    alone, _, _ = v4moe.lora_backward(dy=dy, **q)                              # no shared projection
    close(alone, *expanded(d, e, q["a"], q["ids"], torch.zeros(M, K, device=DEV)), "dx alone")


@pytest.mark.parametrize("count", [1, 40, 900])
def test_a_row_does_not_depend_on_the_others(count):
    torch.manual_seed(count)
    q = inputs(3000, 320, 1000, 24, 11, "any")
    y, dy = rows(3000, 320, t=F32), rows(3000, 320)
    out = v4moe.lora_add(y, **q)
    dx, _, _ = v4moe.lora_backward(dy=dy, dx=torch.empty(3000, 1000, device=DEV), **q)
    some = torch.randperm(3000, device=DEV)[:count]
    p = dict(q, x=q["x"][some].contiguous(), ids=q["ids"][some].contiguous())
    assert torch.equal(v4moe.lora_add(y[some].contiguous(), **p), out[some])
    b, _, _ = v4moe.lora_backward(dy=dy[some].contiguous(), dx=torch.empty(count, 1000, device=DEV), **p)
    assert torch.equal(b, dx[some])


def test_determinism():
    torch.manual_seed(0)
    q = inputs(2500, 256, 512, 32, 5, "any")
    y, dy = rows(2500, 256), rows(2500, 256)
    first = v4moe.lora_add(y, **q), *v4moe.lora_backward(dy=dy, **q)
    for _ in range(5):
        again = v4moe.lora_add(y, **q), *v4moe.lora_backward(dy=dy, **q)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_no_number_keeps_to_its_rows_and_its_adapter():
    torch.manual_seed(1)
    q = inputs(90, 96, 128, 16, 3, "any")
    y, dy = rows(90, 96), rows(90, 96)
    clean = v4moe.lora_add(y, **q), *v4moe.lora_backward(dy=dy, **q)
    bad = int(torch.nonzero(q["ids"] == 1)[0])
    q["x"][bad], dy[bad] = math.nan, math.inf
    q["x"][q["ids"] < 0], dy[q["ids"] < 0] = math.nan, math.nan               # rows without an adapter
    out, (dx, da, db) = v4moe.lora_add(y, **q), v4moe.lora_backward(dy=dy, **q)
    keep = torch.arange(90, device=DEV) != bad
    assert torch.equal(out[keep], clean[0][keep]) and bool(out[bad].isnan().all())
    assert torch.equal(dx[keep], clean[1][keep]) and not bool(dx[bad].isfinite().any())
    for got, was in ((da, clean[2]), (db, clean[3])):
        assert torch.equal(got[[0, 2]], was[[0, 2]]) and bool(got[1].isnan().any())


def test_gradients_against_differences():
    """<dy, out(p + h) - out(p - h)> / 2 = <dp, h>: the result is linear in x, A and B each."""
    torch.manual_seed(2)
    M, N, K, r, L = 20, 24, 40, 5, 3
    q = inputs(M, N, K, r, L, "any")
    y, dy = torch.zeros(M, N, device=DEV), rows(M, N)
    f = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    grads = dict(zip("xab", v4moe.lora_backward(dy=dy, dx=f(M, K), da=f(L, r, K), db=f(L, r, N), **q)))
    for name in "xab":
        step = torch.randint(-1, 2, q[name].shape, device=DEV).to(BF16)
        moved = dict(q, **{name: step})
        want = (dy.double() * v4moe.lora_add(y, **moved).double()).sum()      # linear: the difference over a whole step
        size = dict(moved, **{n: moved[n].abs() for n in "xab"})
        S = float((dy.double().abs() * expanded(factor(size["x"], size["a"], q["ids"], q["scale"])[0] * 1.0,
                                                torch.zeros(M, r, dtype=torch.float64, device=DEV), size["b"], q["ids"], y)[0]).sum())
        got = (grads[name].double() * step.double()).sum()
        # both sides' intermediates to 2^-16, sums of at most 100 terms
        assert abs(float(got - want)) <= 2 * (2.0 ** -16 + 200 * 2.0 ** -23) * S


def test_graph_replays():
    torch.manual_seed(3)
    q = inputs(70, 128, 256, 16, 8, "any")
    y, dy = rows(70, 128), rows(70, 128)

    def step():
        return v4moe.lora_add(y, **q), *v4moe.lora_backward(dy=dy, **q)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        q["x"].copy_(torch.randn_like(q["x"]))
        q["ids"].copy_(torch.randint(-1 - i, 9, (70,), device=DEV))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_beside_the_shared_projection():
    """The path: the FP8 projection, adapters added in place, and both backwards into one dx."""
    torch.manual_seed(4)
    M, N, K = 96, 256, 384
    q = inputs(M, N, K, 16, 6, "any")
    w = v4moe.fp8_weights(torch.randn(N, K, device=DEV) * 0.05)
    shared = v4moe.fp8_linear(q["x"], w)
    out = v4moe.lora_add(shared.clone(), **q)
    want, bound = expanded(*factor(q["x"], q["a"], q["ids"], q["scale"]), q["b"], q["ids"], shared)
    close(out, want, bound, "out")
    dy = rows(M, N)
    dx, _ = v4moe.fp8_linear_backward(q["x"], dy, w)
    both, _, _ = v4moe.lora_backward(dy=dy, base=dx, **q)
    want, bound = expanded(*factor(dy, q["b"], q["ids"], q["scale"]), q["a"], q["ids"], dx)
    close(both, want, bound, "dx")


def test_python_refusals():
    q = inputs(6, 24, 16, 4, 3, "any")
    y, dy = rows(6, 24), rows(6, 24)
    for bad in (dict(x=q["x"].float()), dict(x=q["x"][:, :8]), dict(a=q["a"].float()), dict(a=q["a"][:, :2]), dict(b=q["b"][:2]),
                dict(ids=q["ids"].long()), dict(ids=q["ids"][:5]), dict(scale=q["scale"].double()), dict(scale=q["scale"][:2]),
                dict(y=y[:, :8]), dict(y=y.half()), dict(out=torch.empty(6, 24, device=DEV)), dict(ids=q["ids"].cpu()),
                dict(y=y.cpu()), dict(b=q["b"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            v4moe.lora_add(**{**dict(y=y, **q), **bad})
    for bad in (dict(dy=dy.float()), dict(accumulate=True), dict(base=torch.empty(6, 15, device=DEV)),
                dict(base=torch.empty(6, 16, device=DEV), dx=torch.empty(6, 16, dtype=BF16, device=DEV)),
                dict(da=torch.empty(3, 4, 24, device=DEV)), dict(db=torch.empty(3, 4, 24, dtype=torch.float16, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            v4moe.lora_backward(**{**dict(dy=dy, **q), **bad})
