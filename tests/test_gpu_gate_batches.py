"""moe_gate and moe_gate_backward over large batches of both types inside wider rows, and routing whose every decision
is compared, with and without a bias.

Bars.  Rows of a large batch: forward, in every bit as in a small one; backward, test_gpu_gate.py's.  Decisions: fp32
scores are within 4 units of the last place, 2^-22 relative, a key one rounding more, a group's value the sum of two;
two values whose 64-bit ones differ by 4e-6 of the magnitudes in them (score and bias) are then in the same order.
Equal keys and values (a gap of 0) go by number.  Weights: 2e-6 as in test_gpu_gate.py."""
import itertools

import numpy as np
import pytest
import torch

from fp4_weight_grouped_amd import v4moe
from test_gpu_gate import DEV, NEG, _float32, backward64, logits_of, scores64  # noqa: F401

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# each number of experts per lane and lanes per token that batches from 4096 on take, forward and backward
LAYOUTS = [(20, 3, 1, 1), (32, 6, 8, 3), (45, 5, 15, 6), (64, 7, 16, 4), (72, 6, 8, 3), (128, 16, 8, 4), (96, 6, 32, 9),
           (160, 5, 20, 7), (255, 16, 1, 1), (256, 8, 8, 4), (300, 8, 4, 2)]


def inside(z, ld, at):
    """z as columns at .. of rows of ld elements, the rest NaN."""
    wide = torch.full((z.shape[0], ld), float("nan"), dtype=z.dtype, device=DEV)
    wide[:, at:at + z.shape[1]] = z
    return wide[:, at:at + z.shape[1]]


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("E,k,groups,kept", LAYOUTS)
def test_forward(E, k, groups, kept, type):
    for score, (pad, at) in itertools.product(range(3), ((0, 0), (5, 3), (6, 1))):
        rng = np.random.default_rng([E, k, score, 3])
        z = torch.cat([logits_of(rng, 29, E, type, kind) for kind in ("grid", "ties", "masked")])
        b = (torch.randn(E, device=DEV) * 0.1) if at != 1 else None
        args = dict(score=score, bias=b, groups=groups, topk_groups=kept, renorm=bool(k % 2))
        ids, w = v4moe.gate(z, k, **args)
        many, mw = v4moe.gate(inside(z.repeat(48, 1)[:4105], E + pad, at), k, **args)
        assert torch.equal(many, ids.repeat(48, 1)[:4105]) and torch.equal(mw, w.repeat(48, 1)[:4105]), (score, pad, at)


@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(e, k) for e, k, _, _ in LAYOUTS])
def test_backward(E, k, type):
    """The gradient's rows wider too, through the C entry point: nothing beside its columns is written."""
    for score, renorm, (pad, at) in itertools.product(range(3), (False, True), ((0, 0), (5, 3))):
        backward_of_many(E, k, type, pad, at, renorm, score)


def backward_of_many(E, k, type, pad, at, renorm, score):
    T = 4109
    rng = np.random.default_rng([E, k, score, 5])
    z = torch.cat([logits_of(rng, 31, E, type, kind) for kind in ("grid", "masked")])
    how = dict(score=score, renorm=renorm, scale=2.5)
    ids, w = v4moe.gate(z, k, **how)
    dw = torch.from_numpy(rng.standard_normal((62, k)).astype(np.float32)).to(DEV)
    ref, size = backward64(z.double().cpu().numpy(), ids.cpu().numpy().astype(np.int64), w.cpu().numpy() != 0,
                           dw.cpu().numpy().astype(np.float64), score, renorm, 2.5)
    ref, bar = (np.tile(a, (67, 1))[:T] for a in (ref, 4e-6 * size + (2.0 ** -8 * np.abs(ref) if type == "bf16" else 0) + 1e-30))
    logits = inside(z.repeat(67, 1)[:T], E + pad, at)
    ids, w, dw = (t.repeat(67, 1)[:T].contiguous() for t in (ids, w, dw))
    out = torch.full((T, E + 7), 3.0, dtype=TYPES[type], device=DEV)
    view, P = out[:, 2:E + 2], v4moe._p
    g = v4moe.GateC(T, E, k, score, 1, 1, int(renorm), 2.5)
    code = v4moe.TYPE_BF16 if type == "bf16" else v4moe.TYPE_F32
    assert v4moe.lib().moe_gate_backward(v4moe.ctypes.byref(g), P(logits), code, logits.stride(0), P(ids), P(w), P(dw), P(view),
                                         E + 7, v4moe._stream()) == 0
    assert bool((out[:, :2] == 3).all()) and bool((out[:, E + 2:] == 3).all())
    got = view.double().cpu().numpy()
    assert (np.abs(got - ref) <= bar).all(), np.max(np.abs(got - ref) - bar)
    assert torch.equal(v4moe.gate_backward(logits, ids, w, dw, **how), view)


def decide64(z, k, score, bias, G, kept, renorm, scale):
    """ids, weights and, per token, whether every decision is clear."""
    z, s = scores64(z, score)
    T, E = z.shape
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    ids, w, clear = np.zeros((T, k), np.int64), np.zeros((T, k)), np.ones(T, bool)
    for t in range(T):
        key = np.where((z[t] == NEG) | np.isnan(b), NEG, s[t] + b)
        size = s[t] + np.abs(np.nan_to_num(b, neginf=0.0))

        def order(v, size, n):
            o = sorted(range(len(v)), key=lambda i: (-v[i], i))
            for x, y in zip(o[:n], o[1:n + 1]):
                clear[t] &= v[x] == v[y] or v[x] - v[y] > 4e-6 * max(size[x], size[y])
            return o[:n]

        if G > 1:
            val, vs, n = [], [], E // G
            for g in range(G):
                top = [i for i in sorted(range(g * n, g * n + n), key=lambda i: -key[i])[:2] if key[i] > NEG]
                val.append(sum(key[i] for i in top) if top else NEG)
                vs.append(2 * max((size[i] for i in top), default=0.0))
            keep = order(val, vs, kept)
            key = np.where(np.isin(np.arange(E) // n, keep), key, NEG)
        ids[t] = order(key, size, k)
        p = np.where(key[ids[t]] == NEG, 0, s[t][ids[t]])
        w[t] = scale * (np.where(p.sum() > 0, p / (p.sum() or 1), 0) if renorm else p)
    return ids, w, clear


CASES = [(1, 1, 1, 1, 1), (3, 8, 8, 1, 1), (40, 64, 6, 1, 1), (40, 65, 7, 1, 1), (40, 72, 6, 8, 3), (40, 128, 8, 32, 3),
         (40, 160, 6, 8, 3), (60, 256, 8, 8, 4), (20, 384, 16, 6, 2), (20, 513, 9, 1, 1), (20, 1024, 16, 64, 5), (20, 30, 3, 30, 4)]


def inputs_of(case, kind, biased, score):
    T, E, k, G, kept = case
    rng = np.random.default_rng([E, k, score, int(biased), 11])
    z = np.stack([rng.permutation(np.linspace(-4, 4, E)) for _ in range(T)]).astype(np.float32)
    if kind == "masked":
        z[rng.random((T, E)) < 0.3] = NEG
        z[::4] = NEG
        z[1::4, E // 2:] = np.finfo(np.float32).min
    return z, (rng.integers(-8, 9, E) / 64).astype(np.float32) if biased else None


@pytest.mark.parametrize("kind", ["grid", "masked"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_every_decision(case, kind):
    for biased, score in itertools.product((False, True), range(3)):
        decisions(case, kind, biased, score)


def decisions(case, kind, biased, score):
    T, E, k, G, kept = case
    z, bias = inputs_of(case, kind, biased, score)
    renorm = bool(k % 2)
    ri, rw, clear = decide64(z, k, score, bias, G, kept, renorm, 2.5)
    if kind == "grid" and not biased and G == 1:
        assert clear.all()                   # a grid's gaps
    assert clear.mean() >= 0.8               # (a property of the inputs: 0.85 at the least)
    ids, w = v4moe.gate(torch.from_numpy(z).to(DEV), k, score=score, bias=None if bias is None else torch.from_numpy(bias).to(DEV),
                        groups=G, topk_groups=kept, renorm=renorm, scale=2.5)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert np.array_equal(ids[clear], ri[clear])
    assert np.allclose(w[clear], rw[clear], rtol=2e-6, atol=1e-30)
