"""Refusals of the grouped products, the cross entropy and the adapters: bad arguments are turned away before a
device is touched."""
import ctypes

import pytest
import torch

from fp4_weight_grouped_amd import v4moe

P = ctypes.c_void_p(4096)          # aligned, never dereferenced
MIS = ctypes.c_void_p(4097)
ODD = ctypes.c_void_p(4098)        # aligned to a bf16, not to 16 bytes
ENULL, EDIMS, EALIGN, EWORKSPACE = -1, -2, -3, -4
SIDE = 1 << 22


def call(name, args, **kw):
    assert not set(kw) - set(args)
    return getattr(v4moe.lib(), name)(*dict(args, **kw).values())


# ---- products grouped by expert ----
LINEAR = dict(M=6, E=3, N=16, K=32, x=P, ldx=32, w=P, offsets=P, y=P, y_type=1, ldy=16, ws=P, n=1 << 20, stream=None)
GRADS = dict(M=6, E=3, N=16, K=32, x=P, ldx=32, dy=P, lddy=16, w=P, offsets=P, dx=P, dx_type=1, lddx=32, dw=P, dw_type=0,
             accumulate=0, ws=P, n=1 << 20, stream=None)
SIZES = [dict(M=-1), dict(M=SIDE + 1), dict(E=0), dict(E=1025), dict(N=0), dict(N=SIDE + 1), dict(K=0), dict(K=-5),
         dict(ldx=31), dict(ldx=SIDE + 1)]


@pytest.mark.parametrize("kw", SIZES)
def test_grouped_sizes(kw):
    assert call("moe_grouped_linear", LINEAR, **kw) == EDIMS
    assert call("moe_grouped_linear_backward", GRADS, **kw) == EDIMS


def test_grouped_arguments():
    def f(**kw):
        return call("moe_grouped_linear", LINEAR, **kw)

    assert f(ldy=15) == EDIMS and f(y_type=2) == EDIMS and f(ldy=(1 << 40) + 1) == EDIMS
    assert [f(**{k: None}) for k in ("x", "w", "offsets", "y")] == [ENULL] * 4
    assert [f(**{k: MIS}) for k in ("x", "w", "offsets", "y")] == [EALIGN] * 4
    assert f(y=ODD, y_type=0) == EALIGN and f(offsets=ODD) == EALIGN and f(ws=ODD) == EALIGN
    assert f(M=0, x=None, w=None, offsets=None, y=None, ws=None, n=0) == 0

    def g(**kw):
        return call("moe_grouped_linear_backward", GRADS, **kw)

    assert g(dx=None, dw=None) == ENULL
    assert g(lddy=15) == EDIMS and g(lddx=31) == EDIMS and g(dx_type=-1) == EDIMS and g(dw_type=2) == EDIMS
    assert [g(**{k: None}) for k in ("x", "dy", "w", "offsets")] == [ENULL] * 4
    assert [g(**{k: MIS}) for k in ("x", "dy", "w", "offsets", "dx", "dw")] == [EALIGN] * 6
    assert g(M=0, x=None, dy=None, dw=None) == 0 and g(M=0, x=None, dy=None, accumulate=1) == 0


def test_grouped_workspace():
    def need(M=6, E=3, N=16, K=32, x=P, ldx=32, dy=P, lddy=16, w=P, backward=1):
        return v4moe.lib().moe_grouped_workspace_bytes(M, E, N, K, x, ldx, dy, lddy, w, backward)

    assert need() == 0 and need(backward=0, dy=None, lddy=0) == 0       # everything is read in place
    assert need(M=-1) == need(E=0) == need(K=SIDE + 1) == 0
    assert need(x=ODD) >= 6 * 32 * 2 and need(ldx=33) == need(x=ODD)
    assert need(lddy=17) >= 6 * 16 * 2 and need(lddy=17, backward=0) == 0
    assert need(w=ODD) >= 3 * 16 * 32 * 2
    assert need(K=31, ldx=32) >= 6 * 64 + 3 * 16 * 64
    n = need(K=31, ldx=31, dy=None, lddy=0, backward=0)
    assert call("moe_grouped_linear", LINEAR, K=31, ldx=31, n=n - 1) == EWORKSPACE
    assert call("moe_grouped_linear", LINEAR, K=31, ldx=31, ws=None, n=n) == ENULL
    n = need(lddy=17)
    assert call("moe_grouped_linear_backward", GRADS, lddy=17, n=n - 1) == EWORKSPACE


# ---- cross entropy ----
LOSS = dict(T=5, H=32, V=100, x=P, ldx=32, w=P, ldw=32, targets=P, loss=P, lse=P, ws=P, n=1 << 30, stream=None)
LOSS_GRADS = dict(T=5, H=32, V=100, x=P, ldx=32, w=P, ldw=32, targets=P, lse=P, dloss=P, dloss_stride=1, dx=P, dx_type=1, lddx=32,
                  dw=P, dw_type=0, lddw=32, accumulate=0, ws=P, n=1 << 30, stream=None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=SIDE + 1), dict(H=0), dict(H=SIDE + 1), dict(V=0), dict(V=SIDE + 1), dict(ldx=31),
                                dict(ldw=31), dict(ldw=SIDE + 1)])
def test_xent_sizes(kw):
    assert call("moe_linear_xent", LOSS, **kw) == EDIMS
    assert call("moe_linear_xent_backward", LOSS_GRADS, **kw) == EDIMS


def test_xent_arguments():
    def f(**kw):
        return call("moe_linear_xent", LOSS, **kw)

    assert [f(**{k: None}) for k in ("x", "w", "targets", "loss", "lse", "ws")] == [ENULL] * 6
    assert [f(**{k: MIS}) for k in ("x", "w", "targets", "loss", "lse", "ws")] == [EALIGN] * 6
    assert f(targets=ctypes.c_void_p(4100)) == EALIGN and f(loss=ODD) == EALIGN
    assert f(T=0, x=None, targets=None, loss=None, lse=None, ws=None, n=0) == 0

    def g(**kw):
        return call("moe_linear_xent_backward", LOSS_GRADS, **kw)

    assert g(dx=None, dw=None) == ENULL
    assert g(lddx=31) == EDIMS and g(lddw=31) == EDIMS and g(dx_type=2) == EDIMS and g(dw_type=-1) == EDIMS
    assert g(dloss_stride=-1) == EDIMS and g(dloss_stride=(1 << 40) + 1) == EDIMS
    assert [g(**{k: None}) for k in ("x", "w", "targets", "lse", "dloss", "ws")] == [ENULL] * 6
    assert [g(**{k: MIS}) for k in ("x", "w", "targets", "lse", "dloss", "dx", "dw", "ws")] == [EALIGN] * 8
    assert g(T=0, x=None, targets=None, lse=None, dloss=None, dw=None) == 0
    assert g(T=0, x=None, targets=None, lse=None, dloss=None, accumulate=1) == 0


def test_xent_workspace():
    def need(T=5, H=32, V=100, w=P, ldw=32, backward=1):
        return v4moe.lib().moe_linear_xent_workspace_bytes(T, H, V, w, ldw, backward)

    assert need(T=-1) == need(H=0) == need(V=SIDE + 1) == 0
    for backward in (0, 1):
        n = need(backward=backward)
        assert n > 0 and need(w=ODD, backward=backward) >= n + 100 * 32 * 2
        args = LOSS_GRADS if backward else LOSS
        assert call("moe_linear_xent_backward" if backward else "moe_linear_xent", args, n=n - 1) == EWORKSPACE
    # the logits' gradient: a piece of the vocabulary, not all of it
    assert need(T=8192, H=4096, V=131072) < (1 << 28) + (1 << 28) + 8192 * 4096 * 2
    assert need(T=8192, H=4096, V=131072, backward=0) < 8192 * 4096 * 2 + 8192 * (131072 // 64) * 8 + (1 << 20)


# ---- adapters ----
def sizes(**kw):
    return ctypes.byref(v4moe.LoraC(*dict(dict(M=7, N=16, K=32, r=4, L=3), **kw).values()))


ADD = dict(p=sizes(), y=P, type=1, ldy=16, x=P, ldx=32, a=P, b=P, ids=P, scale=P, out=ctypes.c_void_p(8192), ldo=16, ws=P, n=1 << 20,
           stream=None)
ADD_GRADS = dict(p=sizes(), x=P, ldx=32, dy=P, lddy=16, a=P, b=P, ids=P, scale=P, base=P, ldbase=32, dx=ctypes.c_void_p(8192),
                 dx_type=1, lddx=32, da=P, da_type=0, db=P, db_type=0, accumulate=0, ws=P, n=1 << 20, stream=None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(M=SIDE + 1), dict(N=0), dict(N=SIDE + 1), dict(K=0), dict(K=SIDE + 1), dict(r=0), dict(r=513),
                                dict(L=0), dict(L=65536)])
def test_lora_sizes(kw):
    assert call("moe_lora_add", ADD, p=sizes(**kw)) == EDIMS
    assert call("moe_lora_backward", ADD_GRADS, p=sizes(**kw)) == EDIMS
    assert all(v4moe.lib().moe_lora_workspace_bytes(sizes(**kw), k) == 0 for k in (0, 1))


def test_lora_arguments():
    def f(**kw):
        return call("moe_lora_add", ADD, **kw)

    assert f(p=None) == ENULL and f(ldx=31) == EDIMS and f(ldy=15) == EDIMS and f(ldo=15) == EDIMS and f(type=2) == EDIMS
    assert f(out=P, ldo=17) == EDIMS                                                    # in place with other rows
    assert [f(**{k: None}) for k in ("y", "x", "a", "b", "ids", "scale", "out", "ws")] == [ENULL] * 8
    assert [f(**{k: MIS}) for k in ("y", "x", "a", "b", "ids", "scale", "out", "ws")] == [EALIGN] * 8
    assert f(p=sizes(M=0), y=None, x=None, ids=None, out=None, ws=None, n=0) == 0
    n = v4moe.lib().moe_lora_workspace_bytes(sizes(), 0)
    assert n > 0 and f(n=n - 1) == EWORKSPACE

    def g(**kw):
        return call("moe_lora_backward", ADD_GRADS, **kw)

    assert g(p=None) == ENULL and g(dx=None, da=None, db=None) == ENULL
    assert [g(**{k: 15}) for k in ("ldx", "lddy", "lddx", "ldbase")] == [EDIMS] * 4
    assert [g(**{k: 2}) for k in ("dx_type", "da_type", "db_type")] == [EDIMS] * 3
    assert g(base=ctypes.c_void_p(8192), ldbase=33) == EDIMS
    assert [g(**{k: None}) for k in ("x", "dy", "a", "b", "ids", "scale", "ws")] == [ENULL] * 7
    assert [g(**{k: MIS}) for k in ("x", "dy", "a", "b", "ids", "scale", "base", "dx", "da", "db", "ws")] == [EALIGN] * 11
    assert g(p=sizes(M=0), x=None, dy=None, ids=None, da=None, db=None, ws=None, n=0) == 0
    assert g(p=sizes(M=0), x=None, dy=None, ids=None, accumulate=1, ws=None, n=0) == 0
    n = v4moe.lib().moe_lora_workspace_bytes(sizes(), 1)
    assert n > 0 and g(n=n - 1) == EWORKSPACE


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        v4moe.grouped_linear(x, x[None], torch.zeros(2, dtype=torch.int32))             # not on a GPU
    with pytest.raises(ValueError):
        v4moe.linear_xent(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        v4moe.lora_add(x, x, x[None], x[None], torch.zeros(4, dtype=torch.int32), torch.zeros(1))
    with pytest.raises(ValueError):
        v4moe.lora_add(x, x, x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(1))   # no adapters' axis
