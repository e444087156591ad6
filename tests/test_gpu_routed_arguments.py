"""The layer on a routing the caller made: what the binding turns away before an
address reaches the library, where ids are indices."""
import dataclasses

import numpy as np
import pytest
import torch

from fp4_weight_grouped_amd import inputs, v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, H, I, E, K = 6, 512, 256, 16, 4


@dataclasses.dataclass
class Call:
    layer: v4moe.MoELayer
    x: torch.Tensor
    ids: torch.Tensor
    w: torch.Tensor
    dout: torch.Tensor


@pytest.fixture(scope="module")
def good():
    inp = inputs.make(inputs.Workload("small", inputs.Dims(T=T, H=H, I=I, E=E, topk=K, act=inputs.ACT_SWIGLU)))
    layer = v4moe.MoELayer(H, I, E, K, v4moe.upload_experts(inp.experts, v4moe.dims(T, H, I, E, K), DEV),
                           torch.from_numpy(inp.w_router).to(DEV), DEV)
    x = torch.from_numpy(inp.x.view(np.int16)).to(DEV)
    ids = torch.arange(T * K, dtype=torch.int32, device=DEV).view(T, K) % E
    w = torch.full((T, K), 0.25, dtype=torch.float32, device=DEV)
    return Call(layer, x, ids, w, torch.ones(T, H, dtype=torch.bfloat16, device=DEV))


def strided(t):
    return torch.stack((t, t), dim=-1)[..., 0]


BAD_ROUTING = [dict(ids=lambda t: t.long()), dict(ids=lambda t: t[:-1]), dict(ids=lambda t: t[:, :-1].contiguous()),
               dict(ids=strided), dict(ids=lambda t: t.cpu()), dict(ids=lambda t: t.view(-1)),
               dict(w=lambda t: t.to(torch.bfloat16)), dict(w=lambda t: t.double()), dict(w=lambda t: t[:-1]),
               dict(w=strided), dict(w=lambda t: t.cpu()), dict(x=lambda t: t.float()), dict(x=lambda t: t[:, ::2]),
               dict(x=lambda t: t[:, :H // 2].contiguous()), dict(x=lambda t: t.cpu()), dict(x=lambda t: t.half())]


@pytest.mark.parametrize("bad", BAD_ROUTING, ids=lambda b: next(iter(b)))
def test_routing_and_input(good, bad):
    c = dataclasses.replace(good, **{k: f(getattr(good, k)) for k, f in bad.items()})
    with pytest.raises(ValueError):
        c.layer.forward_routed(c.x, c.ids, c.w)
    with pytest.raises(ValueError):
        c.layer.backward_routed(c.x, c.ids, c.w, c.dout)


def test_outputs(good):
    c = good
    for out in (torch.empty(T, H, device=DEV), torch.empty(T - 1, H, dtype=torch.bfloat16, device=DEV),
                torch.empty(T, 2 * H, dtype=torch.bfloat16, device=DEV)[:, ::2]):
        with pytest.raises(ValueError):
            c.layer.forward_routed(c.x, c.ids, c.w, out=out)
    for dout in (c.dout.float(), c.dout[:-1], strided(c.dout)):
        with pytest.raises(ValueError):
            c.layer.backward_routed(c.x, c.ids, c.w, dout)
    for name in ("dx", "dw", "dWg", "dWu", "dWd"):
        for change in (torch.Tensor.double, lambda t: t[:-1], strided, torch.Tensor.cpu):
            g = c.layer._gradients(T)
            g[name] = change(g[name])
            with pytest.raises(ValueError):
                c.layer.backward_routed(c.x, c.ids, c.w, c.dout, grads=g)
    with pytest.raises(v4moe.V4MoeError):      # what is missing is the library's to refuse
        c.layer.backward_routed(c.x, c.ids, c.w, c.dout, grads=dict(c.layer._gradients(T), dWg=None))


def test_types_of_sixteen_bits(good):
    """The input's and the gradient's bits, whatever 16-bit type carries them."""
    c = good
    out, off = c.layer.forward_routed(c.x, c.ids, c.w)
    grads = c.layer.backward_routed(c.x, c.ids, c.w, c.dout)
    for t in (torch.bfloat16, torch.uint16):
        o, f = c.layer.forward_routed(c.x.view(t), c.ids, c.w, out=torch.empty(T, H, dtype=t, device=DEV))
        assert torch.equal(o.view(torch.int16), out) and torch.equal(f, off)
        g = c.layer.backward_routed(c.x.view(t), c.ids, c.w, c.dout.view(t))
        assert all(torch.equal(g[n], grads[n]) for n in grads)


def test_empty_batch(good):
    e = good.layer.forward_routed(good.x[:0], good.ids[:0], good.w[:0])
    assert e[0].shape == (0, H) and not e[1].any()
