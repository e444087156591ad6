"""Adapters by the thousand: rows are listed by adapter whatever the number of adapters, in passes over the rows where the
list's counters do not hold all of them.

Each row's and each adapter's part of the results is compared with sums in 64 bits (bounds as in the other tests of the
adapters: u and du to 16 bits, fp32 sums of the products), or bit for bit with a call for the adapter alone."""
import ctypes

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
STEP32 = 2.0 ** -23


@pytest.mark.parametrize("L", [16, 1000, 1024, 2047, 2048, 4096, 65535])
def test_gradients_of_many_rows_have_them_listed(L):
    """Without a list every block of an adapter's sums would look through all rows.  (The workspace holds it: the rows' order and
    the tiles beside u and du.)"""
    for M in (1001, 8192):
        p = v4moe.LoraC(M, 64, 64, 16, L)
        u = M * 2 * 16 * 2
        assert v4moe.lib().moe_lora_workspace_bytes(ctypes.byref(p), 1) >= 2 * u + M * 4 + L * 4


def randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(BF16)


def near(got, want, bound):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= bound * (1 + half) + half * want.abs() + 2.0 ** -126)
    assert not bool(bad.any()), (int(bad.sum()), float((got.double() - want).abs().max()))


def per_row(v, f, ids, scale):
    """scale F[id] v of rows with an adapter in 64 bits, and the sums of its products' magnitudes."""
    u, size = (torch.empty(len(ids), f.shape[1], dtype=torch.float64, device=DEV) for _ in range(2))
    for c in range(0, len(ids), 4096):
        k = slice(c, c + 4096)
        q, s = f[ids[k]].double(), scale[ids[k]].double()[:, None]
        u[k] = torch.matmul(q, v[k].double()[:, :, None])[..., 0] * s
        size[k] = torch.matmul(q.abs(), v[k].double().abs()[:, :, None])[..., 0] * s.abs()
    return u, size


# around a pass's 2048 adapters (one more number stands for none), several passes, the most; rows that the list's waves
# hold in registers (8192) and more, fewer than adapters and more, all of one adapter of the last pass
@pytest.mark.gpu
@pytest.mark.parametrize("M,L", [(1500, 1023), (1500, 1024), (1500, 1025), (9000, 2046), (9000, 2047), (9000, 2048), (700, 2049), (8192, 4095),
                                 (8193, 4096), (20000, 6000), (3000, 65535), (66, 65535), (1500, -5000)])
def test_result_and_gradients(M, L):
    torch.set_default_dtype(F32)
    one, L = L < 0, abs(L)                                     # below 0: all rows with the last adapter
    N, K, r = 40, 72, 3
    g = torch.Generator(device=DEV).manual_seed(M + L)
    a, b, x, y, dy = randn(g, L, r, K), randn(g, L, r, N), randn(g, M, K), randn(g, M, N), randn(g, M, N)
    scale = torch.rand(L, generator=g, device=DEV)
    ids = torch.randint(-L // 8 - 1, L + L // 8 + 1, (M,), generator=g, device=DEV).to(torch.int32)
    if one:
        ids[:] = L - 1
    ids[torch.arange(M, device=DEV) % 97 == 5] = L - 1
    ids[torch.arange(M, device=DEV) % 89 == 7] = 0
    at = torch.nonzero((ids >= 0) & (ids < L)).flatten()
    none = (ids < 0) | (ids >= L)
    i = ids.long()[at]
    n = torch.bincount(i, minlength=L).double()[:, None, None]

    out = v4moe.lora_add(y, x, a, b, ids, scale)
    dx, da, db = v4moe.lora_backward(x, dy, a, b, ids, scale, base=x, da=torch.full((L, r, K), 7.0, device=DEV),
                                     db=torch.full((L, r, N), 7.0, device=DEV))
    assert torch.equal(out[none], y[none]) and torch.equal(dx[none], x[none])
    for got, v, f, w, base in ((out, x, a, b, y), (dx, dy, b, a, x)):
        u, size = per_row(v[at], f, i, scale)
        err = size * (v.shape[1] + 64) * STEP32 + u.abs() * (2.0 ** -16 + 2.0 ** -22)
        want, bound = base[at].double(), torch.empty(len(at), w.shape[2], dtype=torch.float64, device=DEV)
        for c in range(0, len(at), 4096):
            k = slice(c, c + 4096)
            q = w[i[k]].double()
            want[k] += torch.matmul(u[k][:, None], q)[:, 0]
            bound[k] = torch.matmul((err[k] + (2 * r + 64) * STEP32 * (u[k].abs() + err[k]))[:, None], q.abs())[:, 0]
        near(got[at], want, bound + STEP32 * want.abs())
    for got, v, f, w in ((da, dy, b, x), (db, x, a, dy)):
        u, size = per_row(v[at], f, i, scale)
        err = size * (v.shape[1] + 64) * STEP32 + u.abs() * (2.0 ** -16 + 2.0 ** -22)
        want, bound, mag = (torch.zeros(got.shape, dtype=torch.float64, device=DEV) for _ in range(3))
        wd = w.double()[at]
        want.index_add_(0, i, u[:, :, None] * wd[:, None])
        bound.index_add_(0, i, err[:, :, None] * wd.abs()[:, None])
        mag.index_add_(0, i, (u.abs() + err)[:, :, None] * wd.abs()[:, None])
        near(got, want, bound + (2 * n + 128) * STEP32 * mag)
        assert not bool(got[n[:, 0, 0] == 0].any())
    # a row alone, and an adapter's rows alone
    k = at[:: max(len(at) // 5, 1)]
    assert torch.equal(out[k], v4moe.lora_add(y[k], x[k], a, b, ids[k], scale))
    assert torch.equal(dx[k], v4moe.lora_backward(x[k], dy[k], a, b, ids[k], scale, base=x[k])[0])
    again = v4moe.lora_backward(x, dy, a, b, ids, scale, base=x, da=torch.empty_like(da), db=torch.empty_like(db))
    assert all(torch.equal(p, q) for p, q in zip((dx, da, db), again))


@pytest.mark.gpu
def test_graph_replays():
    """Captured, with other adapters at each replay."""
    torch.set_default_dtype(F32)
    M, L, N, K, r = 1200, 5000, 64, 64, 4
    g = torch.Generator(device=DEV).manual_seed(1)
    a, b, x, y, dy = randn(g, L, r, K), randn(g, L, r, N), randn(g, M, K), randn(g, M, N), randn(g, M, N)
    scale, ids = torch.rand(L, generator=g, device=DEV), torch.zeros(M, dtype=torch.int32, device=DEV)

    def step():
        return v4moe.lora_add(y, x, a, b, ids, scale), *v4moe.lora_backward(x, dy, a, b, ids, scale)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for most in (L, 3, L + 900, 2049):
        ids.copy_(torch.randint(-2, most, (M,), generator=g, device=DEV))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
