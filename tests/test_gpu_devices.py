"""The operators next to the layer take addresses of the current GPU only: any tensor of another one is refused,
not the first alone."""
import numpy as np
import pytest
import torch

from fp4_weight_grouped_amd import inputs, v4moe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Elsewhere(torch.Tensor):
    """A tensor that says it is on GPU 1 (its memory is on GPU 0: what is not refused still runs)."""

    def get_device(self):
        return 1

    @property
    def device(self):
        return torch.device("cuda", 1)


def there(t):
    return t.as_subclass(Elsewhere)


def bf16(*shape):
    return torch.ones(*shape, dtype=torch.bfloat16, device=DEV)


def f32(*shape):
    return torch.ones(*shape, dtype=torch.float32, device=DEV)


def refused(call, args, moved):
    """call(**args) runs; with any one of the moved arguments elsewhere it does not."""
    call(**args)
    for name in moved:
        with pytest.raises(ValueError, match="GPU 1"):
            call(**dict(args, **{name: there(args[name])}))


def test_gate():
    z, b = f32(4, 16), f32(16)
    refused(lambda logits, bias: v4moe.gate(logits, 2, bias=bias), dict(logits=z, bias=b), ["logits", "bias"])
    ids, w = v4moe.gate(z, 2)
    names = ["logits", "topk_ids", "topk_w", "dw"]
    refused(v4moe.gate_backward, dict(zip(names, (z, ids, w, f32(4, 2)))), names)


def test_fp8_parts():
    refused(v4moe.fp8_quantize, dict(x=f32(4, 32)), ["x"])
    refused(v4moe.fp8_weights, dict(w=f32(4, 32)), ["w"])
    a, b = (torch.zeros(n, 32, dtype=torch.uint8, device=DEV) for n in (4, 8))
    names = ["a", "a_scale", "b", "b_scale", "out"]
    refused(v4moe.fp8_gemm, dict(zip(names, (a, f32(1, 4), b, f32(1, 1), f32(4, 8)))), names)
    refused(v4moe.fp8_gemm, dict(zip(names, (a, f32(1, 4), b, f32(1, 8), f32(4, 8))), rows=True), names)


def test_fp8_linear():
    w = v4moe.fp8_weights(f32(8, 32))

    def forward(x, out, q, qt, blk):
        return v4moe.fp8_linear(x, v4moe.FP8Matrix(8, 32, q, qt, blk), out=out)

    def backward(x, dy, dx, dw, q, qt, blk):
        return v4moe.fp8_linear_backward(x, dy, v4moe.FP8Matrix(8, 32, q, qt, blk), dx=dx, dw=dw)

    m = dict(q=w.q, qt=w.qt, blk=w.blk)
    args = dict(x=bf16(4, 32), out=bf16(4, 8), **m)
    refused(forward, args, args)
    args = dict(x=bf16(4, 32), dy=bf16(4, 8), dx=bf16(4, 32), dw=f32(8, 32), **m)
    refused(backward, args, args)


def test_clip():
    refused(lambda g: v4moe.clip_grads([g], 1.0), dict(g=f32(5)), ["g"])


def test_routed_layer():
    T, H, I, E, k = 4, 512, 256, 8, 2
    inp = inputs.make(inputs.Workload("small", inputs.Dims(T=T, H=H, I=I, E=E, topk=k, act=inputs.ACT_SWIGLU)))
    layer = v4moe.MoELayer(H, I, E, k, v4moe.upload_experts(inp.experts, v4moe.dims(T, H, I, E, k), DEV), None, DEV)
    x = torch.from_numpy(inp.x.view(np.int16)).to(DEV)
    ids, w = v4moe.gate(torch.randn(T, E, dtype=torch.float32, device=DEV), k)
    names = ["d", "x", "topk_ids", "topk_w", "experts", "expert_offsets", "out", "workspace"]
    off, out = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T, H, dtype=torch.int16, device=DEV)
    args = dict(zip(names, (layer.dims(T), x, ids, w, layer.experts, off, out, layer.workspace(T))))
    refused(v4moe.moe_routed_forward, args, ["x", "topk_ids", "topk_w", "expert_offsets", "out", "workspace"])
    g, (wt_gu, wt_d) = layer._gradients(T), layer.transposed_weights()
    args = dict(d=layer.dims(T), x=x, topk_ids=ids, topk_w=w, experts=layer.experts, wt_gu=wt_gu, wt_d=wt_d, dout=bf16(T, H),
                workspace=layer._backward_workspace(layer.dims(T)), **g)
    refused(v4moe.moe_routed_backward, args, [n for n in args if n not in ("d", "experts")])
