"""The operators next to the layer in the paths that use them: the layer with
the routing given, and the example's training steps."""
import os
import sys

import numpy as np
import pytest
import torch

from fp4_weight_grouped_amd import inputs, v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _float32():
    """Other modules set another default type when they are collected."""
    old = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(old)


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def small_layer(T, H=512, I=256, E=16, k=4, act=inputs.ACT_SWIGLU):
    inp = inputs.make(inputs.Workload("small", inputs.Dims(T=T, H=H, I=I, E=E, topk=k, act=act)))
    dims = v4moe.dims(T, H, I, E, k, act)
    layer = v4moe.MoELayer(H, I, E, k, v4moe.upload_experts(inp.experts, dims, DEV), torch.from_numpy(inp.w_router).to(DEV),
                           DEV, act)
    return layer, torch.from_numpy(inp.x.view(np.int16)).to(DEV)


@pytest.mark.parametrize("T", [1, 37, 700])
@pytest.mark.parametrize("act", [inputs.ACT_SWIGLU, inputs.ACT_RELU2])
def test_routing_given_equals_routing_computed(T, act):
    """Every output and gradient bit for bit, at a batch of each router variant and tile."""
    layer, x = small_layer(T, act=act)
    dout = torch.randn(T, layer.H, device=DEV).to(torch.bfloat16)
    out, ids, w, off = layer.forward(x)
    out2, off2 = layer.forward_routed(x, ids, w)
    assert torch.equal(out, out2) and torch.equal(off, off2)
    a = layer.backward(x, dout)
    b = layer.backward_routed(x, ids, w, dout)
    assert a.keys() == b.keys() and all(torch.equal(a[n], b[n]) for n in a)


def test_routing_given_with_masked_tokens():
    """Tokens whose logits are all masked get ids in range and weights 0: a zero output and no gradient of x."""
    T = 64
    layer, x = small_layer(T)
    logits = torch.randn(T, layer.E, device=DEV)
    logits[::3] = -float("inf")
    logits[1::3, : layer.E - 2] = torch.finfo(torch.float32).min
    ids, w = v4moe.gate(logits, layer.topk, groups=4, topk_groups=2)
    out, _ = layer.forward_routed(x, ids, w)
    g = layer.backward_routed(x, ids, w, torch.randn(T, layer.H, device=DEV).to(torch.bfloat16))
    torch.cuda.synchronize()
    y = out.view(torch.bfloat16)
    assert not y[::3].any() and not g["dx"][::3].any()
    assert bool((w[1::3].sum(-1) - 1).abs().max() < 1e-6) and bool(y[1::3].any(dim=1).all())
    assert not v4moe.gate_backward(logits, ids, w, g["dw"])[::3].any()


def test_routed_refusals():
    layer, x = small_layer(4)
    L, d = v4moe.lib(), layer.dims(4)
    ex = layer.experts.c()
    P, ws = v4moe._p, layer.workspace(4)
    ids, w = torch.zeros(4, 4, dtype=torch.int32, device=DEV), torch.zeros(4, 4, device=DEV)
    off, out = torch.empty(17, dtype=torch.int32, device=DEV), torch.empty(4, 512, dtype=torch.int16, device=DEV)
    ref = v4moe.ctypes.byref

    def call(ids=ids, w=w, n=ws.numel()):
        return L.moe_routed_forward(ref(d), P(x), P(ids), P(w), ref(ex), P(off), P(out), P(ws), n, v4moe._stream())

    assert call(ids=None) == -1 and call(w=None) == -1 and call(n=10) == -4
    # the internal mode is not one a caller may pass
    for mode in (-1, 2):
        assert L.moe_layer_forward(ref(d), P(x), P(x), None, mode, None, ref(ex), P(ids), P(w), P(off), P(out), P(ws),
                                   ws.numel(), v4moe._stream()) == -2
        assert L.moe_layer_forward_noalloc(ref(d), P(x), P(x), None, mode, None, ref(ex), P(ids), P(w), P(off), P(out),
                                           v4moe._stream()) == -2


def test_example_trains():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_step
    finally:
        sys.path.pop(0)
    torch.manual_seed(0)
    block = train_step.Block(256, 256, 8, 2, 4, 2)
    a = torch.randn(200, 256, device=DEV).to(torch.bfloat16)
    target = torch.randn(200, 256, device=DEV) * 0.1
    losses, norms = zip(*((float(x), float(n)) for x, n in (block.step(a, target, 4.0, 0.02) for _ in range(8))))
    assert all(np.isfinite(losses)) and all(n > 0 for n in norms)
    assert losses[-1] < 0.9 * losses[0], losses
