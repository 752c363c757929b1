"""The routed experts of a layer from their parts, forward and backward: rows to their experts,
the gate/up product, the gated activation, the down product and the weighted sum back, with
the block-FP8 weights as constants.  What is trained here sits in front of the experts: a
bf16 matrix whose gradient comes through all of them.

    python examples/expert_parts.py [tokens] [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_fp8_mixture_router_gb300 as moe  # noqa: E402
import workloads as W  # noqa: E402


class Experts:
    """The routed half of a layer.  quantize: rows between the products in 8 bits, as the
    layer itself has them; else bf16 rows, which each product quantises on its way."""

    def __init__(self, shape: W.MoEShape, layer: dict, tokens: int, quantize: bool = True):
        self.quantize = quantize
        self.w13 = moe.BlockWeights(layer["w13"], layer["s13"])
        self.w2 = moe.BlockWeights(layer["w2"], layer["s2"])
        self.ops = moe.ExpertOps(shape.n_experts, shape.top_k, tokens,
                                 max(shape.hidden, 2 * shape.inter))

    def forward(self, x: torch.Tensor, idx: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
        """x [tokens, H] by experts idx and weights w [tokens, k]: [tokens, H]."""
        ops, q = self.ops, self.quantize
        self.w = w
        self.order, rows = ops.dispatch(x, idx, quantize=q)
        starts = self.order.starts
        self.gate_up = ops.linear(rows, self.w13, starts=starts)
        self.out = ops.linear(ops.swiglu(self.gate_up, quantize=q), self.w2, starts=starts)
        return ops.combine(self.out, self.order, w)

    def backward(self, dy: torch.Tensor):
        """The gradients of the last forward's x and w."""
        ops, q, starts = self.ops, self.quantize, self.order.starts
        self.dout, dw = ops.combine_grad(dy, self.out, self.order, self.w, quantize=q)
        self.dh = ops.linear_grad(self.dout, self.w2, starts=starts)
        self.dgate_up = ops.swiglu_grad(self.dh, self.gate_up, quantize=q)
        self.drows = ops.linear_grad(self.dgate_up, self.w13, starts=starts)
        return ops.dispatch_grad(self.drows, self.order), dw


def main(tokens: int = 1024, steps: int = 8, shape: W.MoEShape = W.FULL):
    dev = torch.device("cuda", 0)
    torch.cuda.set_device(dev)
    layer = W.make_layer(shape, 1, "bias_skew", device=dev)
    net = moe.MoELayer(moe.LayerShape(shape.hidden, shape.n_experts, shape.top_k, shape.inter,
                                      shape.shared_inter), tokens)
    net.load(layer)
    experts = Experts(shape, layer, tokens)
    x = W.make_x(shape, tokens, 3, "bias_skew", device=dev)
    g = torch.Generator(device=dev).manual_seed(0)
    mix = torch.eye(shape.hidden, device=dev)
    target = 0.05 * torch.randn((tokens, shape.hidden), generator=g, device=dev)
    idx, w = net.route(x)

    def step():
        h = (x.float() @ mix).bfloat16()
        y = experts.forward(h, idx, w)
        error = y.float() - target
        dh, _ = experts.backward(error.bfloat16())
        grad = x.float().t() @ dh.float()
        mix.sub_(grad, alpha=1e-4)
        return error.square().mean(), grad
    a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
    step()
    a.record()
    for _ in range(steps):
        loss, grad = step()
    b.record()
    torch.cuda.synchronize()
    if experts.ops.device_status() != moe.MOE_OK:
        raise RuntimeError("device status flag set")
    assert bool(torch.isfinite(loss)) and bool(torch.isfinite(grad).all())
    print(f"{tokens} tokens, {a.elapsed_time(b) / steps * 1e3:.0f} us a step, "
          f"mean squared error {float(loss):.3e}")


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:3]))
