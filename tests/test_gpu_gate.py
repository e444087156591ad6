"""moe_gate and moe_gate_backward against a plain 64-bit implementation.

Bars.  Ids: equal wherever the 64-bit keys that decide are equal or at least
1e-5 apart (fp32 scores and keys are within a few 2^-24 of theirs, magnitudes up
to about 4).  Weights: fp32 scores are good to a few ulp, the sum of up to 16 and
the division add about one each: 2e-6 relative.  Gradients: products and sums
of up to 16 such terms, each within 2e-6 of the sum of magnitudes; bf16 results
add 2^-9."""
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


NEG = -math.inf


def scores64(z, score):
    z = np.where(np.isnan(z) | (z <= -1e30), NEG, np.minimum(z, 1e30)).astype(np.float64)
    with np.errstate(all="ignore"):
        if score == v4moe.SCORE_SIGMOID:
            return z, 1 / (1 + np.exp(-z))
        if score == v4moe.SCORE_SOFTMAX:
            m = z.max(-1, keepdims=True)
            e = np.exp(z - np.where(m == NEG, 0, m))
            t = e.sum(-1, keepdims=True)
            return z, np.where(t > 0, e / np.where(t > 0, t, 1), 0)
        return z, np.sqrt(np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z))))


def gate64(z, k, score, bias, G, kept, renorm, scale):
    """ids, weights and, per token, whether every decision was clear (a gap of 0 or over 1e-5)."""
    z, s = scores64(z, score)
    T, E = z.shape
    ids, w, clear = np.zeros((T, k), np.int64), np.zeros((T, k)), np.ones(T, bool)
    for t in range(T):
        key = s[t] + (0 if bias is None else bias.astype(np.float64))
        key = np.where((z[t] == NEG) | np.isnan(key), NEG, key)

        def order(v, n):
            o = sorted(range(len(v)), key=lambda i: (-v[i], i))
            for a, b in zip(o[:n], o[1:n + 1]):
                gap = 0.0 if v[a] == v[b] else v[a] - v[b]
                clear[t] &= gap == 0 or gap > 1e-5
            return o[:n]

        if G > 1:
            val = []
            for g in range(G):
                top = sorted(key[g * E // G:(g + 1) * E // G], reverse=True)[:2]
                val.append(top[0] + (top[1] if len(top) > 1 and top[1] > NEG else 0))
            keep = order(val, kept)
            key = np.where(np.isin(np.arange(E) // (E // G), keep), key, NEG)
        ids[t] = order(key, k)
        p = np.where(key[ids[t]] == NEG, 0, s[t][ids[t]])
        w[t] = scale * (np.where(p.sum() > 0, p / (p.sum() or 1), 0) if renorm else p)
    return ids, w, clear


def logits_of(rng, T, E, type, kind):
    """Rows that are permutations of a grid (clear gaps), ties, or masked in places and whole."""
    if kind == "ties":
        z = rng.integers(-2, 3, (T, E)).astype(np.float32)
    else:
        z = np.stack([rng.permutation(np.linspace(-4, 4, E)) for _ in range(T)]).astype(np.float32)
    if kind == "masked":
        low = {"f32": np.finfo(np.float32).min, "bf16": -3.3895313892515355e38}[type]
        z[rng.random((T, E)) < 0.3] = NEG
        z[rng.random((T, E)) < 0.2] = low
        z[rng.random((T, E)) < 0.05] = np.nan
        z[::5] = NEG
        z[1::5] = low
        z[2::5, 1:] = np.nan
        z[3::5, E // 2] = np.inf
    t = torch.from_numpy(z).to(DEV)
    return t.to(torch.bfloat16) if type == "bf16" else t


CASES = [  # T, E, k, groups, kept
    (1, 1, 1, 1, 1), (3, 8, 8, 1, 1), (5, 64, 6, 1, 1), (9, 65, 7, 1, 1), (6, 72, 6, 8, 3), (7, 128, 8, 128 // 4, 3),
    (13, 160, 6, 8, 3), (33, 256, 8, 8, 4), (4, 384, 16, 6, 2), (5, 513, 9, 1, 1), (2, 1024, 16, 64, 5), (3, 40, 5, 20, 7),
    (2, 30, 3, 30, 4), (1030, 256, 8, 8, 4)]


KINDS = [(c, kind, type) for c in CASES for kind in ("grid", "ties", "masked") for type in ("f32", "bf16")
         if c[0] <= 100 or (kind, type) in (("grid", "f32"), ("masked", "bf16"))]


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("case,kind,type", KINDS, ids=str)
def test_forward(case, kind, type, score):
    T, E, k, G, kept = case
    rng = np.random.default_rng([E, k, score])
    z = logits_of(rng, T, E, type, kind)
    bias = None if kind == "ties" else (rng.integers(-8, 9, E) / 64).astype(np.float32)
    if kind == "masked" and E > 4:
        bias[E // 3] = NEG
        bias[E // 4] = np.nan
    renorm, scale = bool(k % 2), 2.5
    ids, w = v4moe.gate(z, k, score=score, bias=None if bias is None else torch.from_numpy(bias).to(DEV), groups=G,
                        topk_groups=kept, renorm=renorm, scale=scale)
    ri, rw, clear = gate64(z.float().cpu().numpy(), k, score, bias, G, kept, renorm, scale)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    if kind == "grid" and type == "f32" and bias is None:
        assert clear.all()
    assert clear.mean() > 0.5 or kind != "ties"
    assert np.array_equal(ids[clear], ri[clear])
    assert np.allclose(w[clear], rw[clear], rtol=2e-6, atol=1e-30)
    for row in ids:
        assert len(set(row)) == k and row.min() >= 0 and row.max() < E


def test_strided_rows_and_stream():
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(rng.standard_normal((50, 100)).astype(np.float32)).to(DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in (torch.float32, torch.bfloat16):
        z = wide.to(t)[:, 3:75]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            ids, w = v4moe.gate(z, 4)
        s.synchronize()
        ids2, w2 = v4moe.gate(z.contiguous(), 4)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_row_does_not_depend_on_the_batch():
    z = torch.randn(700, 256, device=DEV)
    b = torch.randn(256, device=DEV) * 0.1
    for score in range(3):
        ids, w = v4moe.gate(z, 8, score=score, bias=b, groups=8, topk_groups=4)
        for lo, hi in ((0, 1), (5, 8), (600, 700)):
            i2, w2 = v4moe.gate(z[lo:hi], 8, score=score, bias=b, groups=8, topk_groups=4)
            assert torch.equal(ids[lo:hi], i2) and torch.equal(w[lo:hi], w2)


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("kind", ["grid", "ties", "masked"])
@pytest.mark.parametrize("E,k,groups,kept", [(20, 3, 1, 1), (32, 6, 8, 3), (45, 5, 15, 6), (64, 7, 16, 4), (72, 6, 8, 3),
                                             (128, 16, 8, 4), (100, 2, 1, 1), (96, 6, 32, 9), (160, 5, 20, 7),
                                             (256, 8, 8, 4), (255, 16, 1, 1), (300, 8, 4, 2)])
def test_many_tokens(E, k, groups, kept, kind, score):
    """Batches that put several tokens in a wave, the last wave not full: each row as in a small batch, in every bit."""
    rng = np.random.default_rng([E, k, score])
    z = logits_of(rng, 59, E, "f32", kind)
    b = None if kind == "ties" else torch.randn(E, device=DEV) * 0.1
    args = dict(score=score, bias=b, groups=groups, topk_groups=kept, renorm=bool(k % 2))
    ids, w = v4moe.gate(z, k, **args)
    many, mw = v4moe.gate(z.repeat(70, 1)[:4105], k, **args)
    assert torch.equal(many, ids.repeat(70, 1)[:4105]) and torch.equal(mw, w.repeat(70, 1)[:4105])


def weights64(z, ids, live, score, renorm, scale):
    _, s = scores64(z, score)
    p = np.where(live, np.take_along_axis(s, ids, 1), 0)
    if renorm:
        t = p.sum(-1, keepdims=True)
        p = np.where(t > 0, p / np.where(t > 0, t, 1), 0)
    return scale * p


def backward64(z, ids, live, dw, score, renorm, scale):
    zc, s = scores64(z, score)
    T, E = z.shape
    out = np.zeros((T, E))
    size = np.zeros((T, E))
    for t in range(T):
        j = live[t]
        i, d = ids[t][j], dw[t][j]
        p = s[t][i]
        if renorm:
            S = p.sum()
            q = p / S if S > 0 else p * 0
            ds = np.array([scale / S * (q * (a - d)).sum() if S > 0 else 0.0 for a in d])
            mag = np.array([abs(scale) / S * (q * (abs(a) + abs(d))).sum() if S > 0 else 0.0 for a in d])
        else:
            ds, mag = scale * d, np.abs(scale * d)
        if score == v4moe.SCORE_SOFTMAX:
            pe = s[t]
            out[t][i] += ds * p
            size[t][i] += mag * p
            out[t] -= pe * (ds * p).sum()
            size[t] += pe * (mag * p).sum()
        else:
            with np.errstate(all="ignore"):
                f = p * (1 - p) if score == v4moe.SCORE_SIGMOID else np.where(p > 0, 1 / (1 + np.exp(-zc[t][i])) / (2 * np.where(p > 0, p, 1)), 0)
            out[t][i] += ds * f
            size[t][i] += mag * f
    return out, size


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["grid", "masked"])
@pytest.mark.parametrize("case", [(1, 1, 1, 1, 1), (5, 8, 2, 1, 1), (7, 72, 6, 8, 3), (33, 256, 8, 8, 4), (3, 1000, 16, 1, 1)], ids=str)
def test_backward(case, kind, type, renorm, score):
    T, E, k, G, kept = case
    rng = np.random.default_rng([E, k, score, 7])
    z = logits_of(rng, T, E, type, kind)
    if E > 4 and kind == "grid":
        wide = torch.zeros(T, E + 5, dtype=z.dtype, device=DEV)
        wide[:, 2:E + 2] = z
        z = wide[:, 2:E + 2]
    how = dict(score=score, renorm=renorm, scale=2.5)
    ids, w = v4moe.gate(z, k, groups=G, topk_groups=kept, **how)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(DEV)
    dl = v4moe.gate_backward(z, ids, w, dw, **how)
    assert dl.dtype == z.dtype
    zn, idn, live = z.float().cpu().numpy().astype(np.float64), ids.cpu().numpy().astype(np.int64), w.cpu().numpy() != 0
    dwn = dw.cpu().numpy().astype(np.float64)
    ref, size = backward64(zn, idn, live, dwn, score, renorm, 2.5)
    got = dl.float().cpu().numpy()
    bar = 4e-6 * size + (2.0 ** -8 * np.abs(ref) if type == "bf16" else 0) + 1e-30
    assert (np.abs(got - ref) <= bar).all(), np.max(np.abs(got - ref) - bar)
    if kind == "grid" and type == "f32":
        # against differences of the weights, the picks held fixed
        h = 1e-6
        for e in rng.integers(0, E, 6):
            up, dn = zn.copy(), zn.copy()
            up[:, e] += h
            dn[:, e] -= h
            d = ((weights64(up, idn, live, score, renorm, 2.5) - weights64(dn, idn, live, score, renorm, 2.5)) * dwn).sum(-1) / (2 * h)
            assert np.allclose(got[:, e], d, rtol=1e-4, atol=1e-6)


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,k", [(20, 3), (32, 1), (45, 5), (64, 16), (72, 6), (128, 8), (160, 16), (256, 8), (255, 7), (300, 4)])
def test_backward_many_tokens(E, k, renorm, score):
    """Several tokens in a wave, the last wave not full: every row to the bar of the small batch."""
    rng = np.random.default_rng([E, k, score, 9])
    z = logits_of(rng, 61, E, "f32", "masked")
    z[:20] = logits_of(rng, 20, E, "f32", "grid")
    how = dict(score=score, renorm=renorm, scale=2.5)
    ids, w = v4moe.gate(z, k, **how)
    dw = torch.from_numpy(rng.standard_normal((61, k)).astype(np.float32)).to(DEV)
    many = [t.repeat(68, 1)[:4109].contiguous() for t in (z, ids, w, dw)]
    got = v4moe.gate_backward(*many, **how).cpu().numpy()
    ref, size = backward64(z.cpu().numpy().astype(np.float64), ids.cpu().numpy().astype(np.int64), w.cpu().numpy() != 0,
                           dw.cpu().numpy().astype(np.float64), score, renorm, 2.5)
    ref, bar = (np.tile(a, (68, 1))[:4109] for a in (ref, 4e-6 * size + 1e-30))
    assert (np.abs(got - ref) <= bar).all(), np.max(np.abs(got - ref) - bar)


def test_empty():
    z = torch.zeros(0, 16, device=DEV)
    ids, w = v4moe.gate(z, 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert v4moe.gate_backward(z, ids, w, w).shape == (0, 16)
