"""moe_gate_backward where the picked scores are tiny but their shares are not (sums of scores near and below
fp32's smallest normal number), and where a score's derivative is.

Bars.  As in test_gpu_gate.py, 4e-6 of the sum of magnitudes, plus what the subnormal steps of the score leave:
exp(z) is held to two steps, 2^-148, so softplus and a sigmoid this small to d = 2^-148 / exp(z) relative, and the
square root to less; a share s / S is then off by at most 2 d (its own and the sum's), and the sum over shares
times a share by 4 d."""
import itertools
import math

import numpy as np
import pytest
import torch

from fp4_weight_grouped_amd import v4moe
from test_gpu_gate import DEV, _float32, scores64, weights64  # noqa: F401

pytestmark = pytest.mark.gpu

LOW = {v4moe.SCORE_SIGMOID: (-88.7, -88.4), v4moe.SCORE_SQRTSOFTPLUS: (-97.0, -88.8)}
ROWS = {"low": lambda lo, hi: (lo, hi), "normal": lambda lo, hi: (-80.0, -60.0), "middle": lambda lo, hi: (-17.0, -15.0),
        "mixed": lambda lo, hi: (lo, 30.0)}


def gradient64(z, ids, live, dw, score, renorm, scale):
    """The gradient at the picked logits, and the sum of magnitudes: share times the score's logarithmic derivative,
    each in a form that does not cancel."""
    _, s = scores64(z, score)
    s = np.where(live, np.take_along_axis(s, ids, 1), 0)
    zj = np.take_along_axis(z, ids, 1)
    f = 1 / (1 + np.exp(zj))
    if score == v4moe.SCORE_SQRTSOFTPLUS:
        f = 0.5 / (1 + np.exp(-zj)) / np.logaddexp(zj, 0)
    if renorm:
        q = s / s.sum(axis=1, keepdims=True)
        d = (q[:, None, :] * (dw[:, :, None] - dw[:, None, :])).sum(axis=2)
        mag = (q[:, None, :] * (abs(dw[:, :, None]) + abs(dw[:, None, :]))).sum(axis=2)
    else:
        q, d, mag = s, dw, abs(dw)
    out, size = np.zeros_like(z), np.zeros_like(z)
    np.put_along_axis(out, ids, np.where(live, scale * d * q * f, 0), 1)
    np.put_along_axis(size, ids, np.where(live, scale * mag * q * f, 0), 1)
    return out, size


@pytest.mark.parametrize("score", list(LOW))
@pytest.mark.parametrize("rows", list(ROWS))
def test_small_scores(rows, score):
    for k, renorm, T in itertools.product((2, 5), (True, False), (7, 4100)):
        gradient(rows, score, k, renorm, T)


def gradient(rows, score, k, renorm, T):
    E, scale = 24, 8.0
    lo, hi = ROWS[rows](*LOW[score])
    rng = np.random.default_rng([score, k, T])
    z7 = np.stack([rng.permutation(np.linspace(lo, hi, E)) for _ in range(7)]).astype(np.float32)
    z = torch.from_numpy(z7).to(DEV)
    how = dict(score=score, renorm=renorm, scale=scale)
    ids, w = v4moe.gate(z, k, **how)
    dw = torch.from_numpy(rng.standard_normal((7, k)).astype(np.float32)).to(DEV)
    n = -(-T // 7)
    got = v4moe.gate_backward(*(t.repeat(n, 1)[:T].contiguous() for t in (z, ids, w, dw)), **how).cpu().numpy()
    assert np.isfinite(got).all()
    z64, idn, live, dwn = (z7.astype(np.float64), ids.cpu().numpy().astype(np.int64), w.cpu().numpy() != 0,
                           dw.cpu().numpy().astype(np.float64))
    assert live.all()
    ref, size = gradient64(z64, idn, live, dwn, score, renorm, scale)
    smallest = np.take_along_axis(z64, idn, 1).min(axis=1, keepdims=True)
    bar = (4e-6 + 4 * 2.0 ** -148 / np.exp(smallest)) * size + 2.0 ** -148
    ref, bar = (np.tile(a, (n, 1))[:T] for a in (ref, bar))
    assert (np.abs(got - ref) <= bar).all(), np.max((np.abs(got - ref) - bar) / (np.abs(ref) + 1e-300))
    if renorm:
        # against differences of the weights, the picks held fixed; sums of 4 d of magnitudes about 1
        h = 1e-6
        d = 4 * 2.0 ** -148 / math.exp(smallest.min())
        for e in range(0, E, 5):
            up, dn = z64.copy(), z64.copy()
            up[:, e] += h
            dn[:, e] -= h
            diff = ((weights64(up, idn, live, score, renorm, scale) - weights64(dn, idn, live, score, renorm, scale)) * dwn).sum(-1) / (2 * h)
            assert np.allclose(got[:7, e], diff, rtol=1e-4, atol=1e-6 + d * scale * 2 * np.abs(dwn).max())
