"""Training steps of a block on one GPU: a dense projection in FP8, a gate, the FP4 experts, all with their
gradients, and one clipping over everything.

    a -> h = FP8 projection(a) -> logits = h W_r -> gate (sigmoid, balance bias, groups) -> experts(h) -> y

Master weights are fp32.  Each step quantises them (experts to MXFP4, the projection to E4M3 with 128x128 block
scales), runs forward and backward, clips the joint norm of all gradients and takes a step of plain gradient
descent; the gate's bias moves against the experts' load, outside the gradients.  Run it from the repository's root:

    python examples/train_step.py [--steps 20] [--tokens 512] [--hidden 512] [--inner 256] [--experts 32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp4_weight_grouped_amd import v4moe  # noqa: E402


class Block:
    def __init__(self, hidden: int, inner: int, experts: int, topk: int, groups: int, topk_groups: int, seed: int = 0,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

        self.topk, self.groups, self.topk_groups = topk, groups, topk_groups
        self.how = dict(score=v4moe.SCORE_SIGMOID, renorm=True, scale=1.0)
        self.master = dict(projection=weight(hidden, hidden), router=weight(experts, hidden).t().contiguous(),
                           gate=weight(experts, inner, hidden), up=weight(experts, inner, hidden),
                           down=weight(experts, hidden, inner))
        self.bias = torch.zeros(experts, device=device)
        self.layer = v4moe.MoELayer(hidden, inner, experts, topk, None, None, device)
        self.quantise()

    def quantise(self):
        m = self.master
        self.projection = v4moe.fp8_weights(m["projection"])
        self.layer.set_experts(v4moe.DeviceExperts(*(v4moe.quantize_weights(m[k], packed=True) for k in ("gate", "up", "down"))))

    def forward(self, a: torch.Tensor):
        """a: bf16 [T][H].  Returns (y bf16 [T][H], what the backward needs)."""
        h = v4moe.fp8_linear(a, self.projection)
        logits = h.float() @ self.master["router"]
        ids, w = v4moe.gate(logits, self.topk, bias=self.bias, groups=self.groups, topk_groups=self.topk_groups, **self.how)
        y, offsets = self.layer.forward_routed(h, ids, w)
        return y.view(torch.bfloat16), (a, h, logits, ids, w, offsets)

    def backward(self, saved, dy: torch.Tensor) -> dict:
        """Gradients of the master weights from dy = dL/dy (bf16)."""
        a, h, logits, ids, w, _ = saved
        g = self.layer.backward_routed(h, ids, w, dy)
        dlogits = v4moe.gate_backward(logits, ids, w, g["dw"], **self.how)
        dh = g["dx"] + dlogits @ self.master["router"].t()
        dp = torch.empty_like(self.master["projection"])
        v4moe.fp8_linear_backward(a, dh, self.projection, dw=dp)
        return dict(projection=dp, router=h.float().t() @ dlogits, gate=g["dWg"], up=g["dWu"], down=g["dWd"])

    def step(self, a: torch.Tensor, target: torch.Tensor, lr: float, max_norm: float):
        """One step on the mean squared error to target.  Returns (loss, gradient norm) on the GPU."""
        y, saved = self.forward(a)
        error = y.float() - target
        grads = self.backward(saved, (error * (2.0 / error.numel())).to(torch.bfloat16))
        norm = v4moe.clip_grads(grads.values(), max_norm)
        for name, grad in grads.items():
            self.master[name].sub_(grad, alpha=lr)
        load = saved[-1].diff().float()                     # pairs per expert
        self.bias += 0.001 * torch.sign(load.mean() - load)
        self.quantise()
        return error.square().mean(), norm


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inner", type=int, default=256)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--groups", type=int, default=4)
    ap.add_argument("--topk-groups", type=int, default=2)
    ap.add_argument("--lr", type=float, default=4.0)
    ap.add_argument("--max-norm", type=float, default=0.02)
    c = ap.parse_args()
    block = Block(c.hidden, c.inner, c.experts, c.topk, c.groups, c.topk_groups)
    a = torch.randn(c.tokens, c.hidden, device="cuda").to(torch.bfloat16)
    target = torch.randn(c.tokens, c.hidden, device="cuda") * 0.1
    for i in range(c.steps):
        loss, norm = block.step(a, target, c.lr, c.max_norm)
        print(f"step {i}: loss {float(loss):.5f}  gradient norm {float(norm):.4f}", flush=True)


if __name__ == "__main__":
    main()
