"""moe_clip_grads turns away lists whose written memory overlaps another entry's, before a device is touched."""
import ctypes
import math
import random

import pytest

from fp4_weight_grouped_amd import v4moe

EDIMS, EWORKSPACE = -2, -4
F32, BF16 = v4moe.TYPE_F32, v4moe.TYPE_BF16
P = ctypes.c_void_p(4096)          # aligned, never dereferenced


def call(entries, max_norm=1.0):
    """The answer to a list of (g, out, n, type) with a workspace of no bytes: EWORKSPACE once the list is accepted."""
    t = (v4moe.TensorC * len(entries))(*(v4moe.TensorC(*e) for e in entries))
    return v4moe.lib().moe_clip_grads(len(entries), t, max_norm, P, P, 0, None)


@pytest.mark.parametrize("entries", [
    [(4096, 0, 8, F32), (4096, 0, 8, F32)],                           # one gradient listed twice, in place
    [(4096, 4096, 8, F32), (4096, 0, 8, F32)],
    [(4096, 0, 8, F32), (4124, 0, 8, F32)],                           # the last element of the first
    [(8192, 4096, 8, F32), (12288, 4096, 8, F32)],                    # one output of two gradients
    [(8192, 4096, 8, F32), (4126, 12288, 8, BF16)],                   # an output over another gradient
    [(4096, 4100, 8, F32)],                                           # an output shifted over its own gradient
    [(1 << 20, 0, 1 << 20, BF16), (1 << 19, 0, 4, F32), ((1 << 20) + 2048, 0, 4, F32)]])
def test_refused(entries):
    for order in (entries, entries[::-1]):
        assert call(order) == EDIMS
        # among many others
        far = [((1 << 30) + 4096 * i, 0, 1024, F32) for i in range(200)]
        assert call(far[:100] + order + far[100:]) == EDIMS


@pytest.mark.parametrize("entries", [
    [(4096, 0, 8, F32), (4128, 0, 8, F32)],                           # neighbours
    [(4096, 8192, 8, F32), (4096, 12288, 8, F32)],                    # one gradient into two outputs
    [(4096, 0, 0, F32), (4096, 0, 8, F32), (4096, 0, 0, F32)],        # nothing of no elements
    [(4096, 4096, 8, F32)]])
def test_accepted(entries):
    for order in (entries, entries[::-1]):
        assert call(order) == EWORKSPACE


def test_norm_alone():
    """An infinite max_norm writes nothing in place: any list may be counted."""
    assert call([(4096, 0, 8, F32), (4096, 0, 8, F32)], math.inf) == EWORKSPACE
    assert call([(4096, 0, 8, F32), (4100, 8192, 8, F32)], math.inf) == EWORKSPACE
    assert call([(4096, 0, 8, F32), (12288, 4096, 8, F32)], math.inf) == EDIMS


def test_against_pairs():
    """Random lists against the definition, pair by pair."""
    rng = random.Random(0)
    seen = {EDIMS: 0, EWORKSPACE: 0}
    for _ in range(2000):
        entries = [(4096 + 4 * rng.randrange(400), rng.choice((0, 4096 + 4 * rng.randrange(400))), rng.randrange(12), rng.choice((F32, BF16)))
                   for _ in range(rng.randrange(1, 7))]
        ranges = []
        for i, (g, out, n, type) in enumerate(entries):
            size = n * (4 if type == F32 else 2)
            ranges.append((g, g + size, out in (0, g)))
            if out not in (0, g):
                ranges.append((out, out + size, True))
        bad = any((a[2] or b[2]) and a[0] < b[1] and b[0] < a[1] and a[0] < a[1] and b[0] < b[1]
                  for i, a in enumerate(ranges) for b in ranges[:i])
        want = EDIMS if bad else EWORKSPACE
        assert call(entries) == want, entries
        seen[want] += 1
    assert min(seen.values()) > 200
