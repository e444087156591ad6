"""Refusals of the operators next to the layer (gating, FP8 products, clipping):
bad arguments are turned away before a device is touched."""
import ctypes

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

P = ctypes.c_void_p(4096)          # aligned, never dereferenced
MIS = ctypes.c_void_p(4097)
ENULL, EDIMS, EALIGN, EWORKSPACE = -1, -2, -3, -4


def gate(**kw):
    d = dict(T=4, E=64, topk=4, score=0, groups=1, topk_groups=1, renorm=1, scale=1.0)
    d.update(kw)
    return v4moe.GateC(*d.values())


@pytest.mark.parametrize("kw", [dict(T=-1), dict(E=0), dict(E=1025), dict(topk=0), dict(topk=17), dict(E=3),
                                dict(score=3), dict(score=-1), dict(groups=0), dict(groups=65, E=65), dict(groups=7),
                                dict(groups=8, topk_groups=9), dict(topk_groups=0), dict(groups=32, topk_groups=1)])
def test_gate_dims(kw):
    L = v4moe.lib()
    g = gate(**kw)
    assert L.moe_gate(ctypes.byref(g), P, 0, 2000, None, P, P, None) == EDIMS
    assert L.moe_gate_backward(ctypes.byref(g), P, 0, 2000, P, P, P, P, 2000, None) == EDIMS


def test_gate_pointers():
    L = v4moe.lib()
    g = ctypes.byref(gate())
    assert L.moe_gate(None, P, 0, 64, None, P, P, None) == ENULL
    assert L.moe_gate(g, None, 0, 64, None, P, P, None) == ENULL
    assert L.moe_gate(g, P, 0, 64, None, None, P, None) == ENULL
    assert L.moe_gate(g, P, 0, 63, None, P, P, None) == EDIMS
    assert L.moe_gate(g, P, 2, 64, None, P, P, None) == EDIMS
    assert L.moe_gate(g, MIS, 0, 64, None, P, P, None) == EALIGN
    assert L.moe_gate(g, MIS, 1, 64, None, P, P, None) == EALIGN
    assert L.moe_gate(g, P, 0, 64, MIS, P, P, None) == EALIGN
    assert L.moe_gate(ctypes.byref(gate(T=0)), None, 0, 64, None, None, None, None) == 0
    assert L.moe_gate_backward(g, P, 0, 64, P, P, P, P, 63, None) == EDIMS
    assert L.moe_gate_backward(g, P, 0, 64, P, P, None, P, 64, None) == ENULL
    assert L.moe_gate_backward(g, P, 0, 64, P, P, P, MIS, 64, None) == EALIGN


def test_fp8_quantize():
    L = v4moe.lib()
    assert L.moe_fp8_quantize(-1, 16, P, 0, 16, P, P, None, None, None) == EDIMS
    assert L.moe_fp8_quantize(16, (1 << 22) + 1, P, 0, 1 << 23, P, P, None, None, None) == EDIMS
    assert L.moe_fp8_quantize(16, 16, P, 0, 15, P, P, None, None, None) == EDIMS
    assert L.moe_fp8_quantize(16, 16, P, 5, 16, P, P, None, None, None) == EDIMS
    assert L.moe_fp8_quantize(16, 16, None, 0, 16, P, P, None, None, None) == ENULL
    assert L.moe_fp8_quantize(16, 16, P, 0, 16, P, None, None, None, None) == ENULL
    assert L.moe_fp8_quantize(16, 16, P, 0, 16, None, None, None, None, None) == ENULL
    assert L.moe_fp8_quantize(16, 16, P, 0, 16, None, None, MIS, P, None) == EALIGN
    assert L.moe_fp8_quantize(0, 16, None, 0, 16, P, P, None, None, None) == 0
    assert L.moe_fp8_quantize_weights(0, 16, P, 0, 16, P, P, P, None) == EDIMS
    assert L.moe_fp8_quantize_weights(16, 16, P, 0, 16, P, None, P, None) == ENULL
    assert L.moe_fp8_quantize_weights(16, 16, P, 0, 16, MIS, P, P, None) == EALIGN


def gemm(**kw):
    d = dict(M=4, N=8, K=32, b_scale=0, c_type=1, accumulate=0, lda=32, ldb=32, ldc=8, bs_n=1, bs_k=1)
    d.update(kw)
    return v4moe.GemmC(*d.values())


@pytest.mark.parametrize("kw", [dict(M=-1), dict(N=(1 << 22) + 1), dict(K=33), dict(K=17), dict(lda=16), dict(lda=40),
                                dict(ldb=40), dict(lda=1 << 23), dict(b_scale=2), dict(c_type=2), dict(ldc=7)])
def test_fp8_gemm_dims(kw):
    g = gemm(**kw)
    assert v4moe.lib().moe_fp8_gemm(ctypes.byref(g), P, P, P, P, P, None) == EDIMS


def test_fp8_gemm_pointers():
    L, g = v4moe.lib(), ctypes.byref(gemm())
    assert L.moe_fp8_gemm(None, P, P, P, P, P, None) == ENULL
    for i in range(5):
        a = [P] * 5
        a[i] = None
        assert L.moe_fp8_gemm(g, *a, None) == ENULL
        a[i] = MIS
        assert L.moe_fp8_gemm(g, *a, None) == EALIGN
    assert L.moe_fp8_gemm(ctypes.byref(gemm(M=0)), None, None, None, None, None, None) == 0


def test_fp8_linear():
    L = v4moe.lib()
    n = L.moe_fp8_linear_workspace_bytes(4, 8, 32, 0)
    nb = L.moe_fp8_linear_workspace_bytes(4, 8, 32, 1)
    assert n >= 4 * 32 + 4 * 4 and nb > 0
    assert L.moe_fp8_linear_workspace_bytes(4, 0, 32, 0) == 0
    assert L.moe_fp8_linear_workspace_bytes(-1, 8, 32, 1) == 0
    w = v4moe.FP8MatC(8, 32, 4096, 4096, 4096)
    assert L.moe_fp8_linear(4, P, 1, 32, None, P, 1, 8, P, n, None) == ENULL
    assert L.moe_fp8_linear(4, P, 1, 31, ctypes.byref(w), P, 1, 8, P, n, None) == EDIMS
    assert L.moe_fp8_linear(4, P, 1, 32, ctypes.byref(w), P, 1, 7, P, n, None) == EDIMS
    assert L.moe_fp8_linear(4, P, 1, 32, ctypes.byref(w), P, 1, 8, None, n, None) == ENULL
    assert L.moe_fp8_linear(4, P, 1, 32, ctypes.byref(w), P, 1, 8, MIS, n, None) == EALIGN
    assert L.moe_fp8_linear(4, P, 1, 32, ctypes.byref(w), P, 1, 8, P, n - 1, None) == EWORKSPACE
    assert L.moe_fp8_linear(4, P, 1, 32, ctypes.byref(v4moe.FP8MatC(8, 32, 0, 0, 4096)), P, 1, 8, P, n, None) == ENULL
    b = ctypes.byref(w)
    assert L.moe_fp8_linear_backward(4, P, 1, 32, P, 1, 8, b, None, 1, 32, None, 1, 32, 0, P, nb, None) == ENULL
    assert L.moe_fp8_linear_backward(4, P, 1, 32, P, 1, 8, b, P, 1, 32, P, 1, 31, 0, P, nb, None) == EDIMS
    assert L.moe_fp8_linear_backward(4, P, 1, 32, P, 1, 8, b, P, 1, 32, P, 1, 32, 0, P, nb - 1, None) == EWORKSPACE
    noqt = ctypes.byref(v4moe.FP8MatC(8, 32, 4096, 0, 4096))
    assert L.moe_fp8_linear_backward(4, P, 1, 32, P, 1, 8, noqt, P, 1, 32, P, 1, 32, 0, P, nb, None) == ENULL


def test_clip():
    L = v4moe.lib()
    n = L.moe_clip_workspace_bytes(3)
    assert n > 0 and L.moe_clip_workspace_bytes(-1) == 0 and L.moe_clip_workspace_bytes((1 << 20) + 1) == 0

    def call(t, count=1, max_norm=1.0, norm=P, ws=P, size=n):
        return L.moe_clip_grads(count, t, max_norm, norm, ws, size, None)

    def one(g=4096, out=4096, n=8, type=0):
        return (v4moe.TensorC * 1)(v4moe.TensorC(g, out, n, type))

    assert call(None) == ENULL
    assert call(one(), count=-1) == EDIMS
    assert call(one(n=-1)) == EDIMS
    assert call(one(n=(1 << 36) + 1)) == EDIMS
    assert call(one(type=2)) == EDIMS
    assert call(one(g=0)) == ENULL
    assert call(one(g=4098)) == EALIGN
    assert call(one(out=4097, type=1)) == EALIGN
    assert call(one(), max_norm=-1.0) == EDIMS
    assert call(one(), max_norm=float("nan")) == EDIMS
    assert call(one(), norm=None) == ENULL
    assert call(one(), ws=MIS) == EALIGN
    assert call(one(), size=n - 1) == EWORKSPACE


def test_binding_refuses():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        v4moe.gate(x, 2)                       # not on a GPU
    with pytest.raises(ValueError):
        v4moe.fp8_weights(x)
    with pytest.raises(ValueError):
        v4moe.clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        v4moe.clip_grads([], 1.0)
