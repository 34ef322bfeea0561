#!/usr/bin/env python3
"""A feed-forward block that keeps its activations in 8 bits for the backward pass and
serves with weights and tokens in 8-bit integers.

    python examples/eight_bit_block.py [--width 4096] [--hidden 16384] [--tokens 2048] [--steps 20]

    h = x + r;  y = layer_norm(h);  p = y W1 + b1;  out = gelu(p) W2 + b2 + h

Training keeps h, the rows of y and of p in 8-bit floats with a scale each, and nothing
else: gelu(p), the second product's operand, is made again from p. One byte per value of
the hidden layer where the block in 16 bits keeps four (p and gelu(p)). Serving quantizes
the tokens row by row (the norm writes them so) against weights with a scale per output;
a single token's step is captured in a CUDA graph. Data and weights are synthetic.
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_gemm_gb300 import layer_norm, layer_norm_backward, linear, linear_backward, quantize_rows
from examples.mlp_block import captured, microseconds, train


class Block(torch.autograd.Function):
    """out and h of x, the residual stream r and the block's parameters; W1 and W2 kept as [out, in]."""

    @staticmethod
    def forward(ctx, x, r, gain, shift, w1, b1, w2, b2):
        n = layer_norm(x, gain, shift, residual=r, return_stats=True)
        u, p = linear(n.y, w1.t(), b1, activation="gelu", return_pre=True)
        out = linear(u, w2.t(), b2, residual=n.h)
        y8, y_scale = quantize_rows(n.y)
        p8, p_scale = quantize_rows(p)
        ctx.save_for_backward(n.h, n.mean, n.rstd, y8, y_scale, p8, p_scale, gain, w1, w2)
        return out

    @staticmethod
    def backward(ctx, grad):
        h, mean, rstd, y8, y_scale, p8, p_scale, gain, w1, w2 = ctx.saved_tensors
        grad = grad.contiguous()
        du, dw2, db2 = linear_backward(grad, p8, w2.t(), scale_a=p_scale, activation_a="gelu", need_bias=True)
        dy, dw1, db1 = linear_backward(du, y8, w1.t(), scale_a=y_scale, pre=p8, scale_pre=p_scale, activation="gelu", need_bias=True)
        dx, dgain, dshift = layer_norm_backward(dy, h, gain, mean, rstd, grad_h=grad)
        return dx, dx, dgain.to(gain.dtype), dshift.to(gain.dtype), dw1.t(), db1, dw2.t(), db2


class EightBitBlock(torch.nn.Module):
    def __init__(self, width, hidden, dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(out, into):
            return torch.nn.Parameter((torch.randn(out, into, generator=g, device=device) * into ** -0.5).to(dtype))

        self.gain = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        self.shift = torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype))
        self.w1, self.b1 = weight(hidden, width), torch.nn.Parameter(torch.zeros(hidden, device=device))
        self.w2, self.b2 = weight(width, hidden), torch.nn.Parameter(torch.zeros(width, device=device))

    def forward(self, x, r):
        """The block's output (the next residual stream) for x [tokens, width] and r; differentiable."""
        return Block.apply(x, r, self.gain, self.shift, self.w1, self.b1, self.w2, self.b2)

    @torch.no_grad()
    def serve(self, x, r):
        """The same without what the gradients need."""
        n = layer_norm(x, self.gain, self.shift, residual=r)
        u = linear(n.y, self.w1.t(), self.b1, activation="gelu")
        return linear(u, self.w2.t(), self.b2, residual=n.h)


class IntegerBlock:
    """``EightBitBlock.serve`` with both weights in 8-bit integers, a scale per output."""

    @torch.no_grad()
    def __init__(self, block):
        self.block = block
        self.w1, self.s1 = quantize_rows(block.w1, torch.int8)
        self.w2, self.s2 = quantize_rows(block.w2, torch.int8)

    @torch.no_grad()
    def serve(self, x, r):
        b = self.block
        n = layer_norm(x, b.gain, b.shift, residual=r, out_dtype=torch.int8)
        u = linear(n.y, self.w1.t(), b.b1, activation="gelu", scale_a=n.scale, scale_b=self.s1, out_dtype=x.dtype)
        q, scale = quantize_rows(u, torch.int8)
        return linear(q, self.w2.t(), b.b2, residual=n.h, scale_a=scale, scale_b=self.s2)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=16384)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    block = EightBitBlock(a.width, a.hidden)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, target = (torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16() for _ in range(3))
    losses = train(block, x, r, target.float(), a.steps)
    print(f"trained {a.steps} steps on {a.tokens} tokens: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    low = IntegerBlock(block)
    full, eight = block.serve(x, r).float(), low.serve(x, r).float()
    print(f"8-bit integers: relative difference of the block's output {float((eight - full).norm() / full.norm()):.4f}")
    for name, serve in (("16-bit", block.serve), ("8-bit integers", low.serve)):
        graph = captured(serve, x[:1], r[:1])[0]
        print(f"{name}: {microseconds(graph):.1f} us for one token (weights may stay in L2)")


if __name__ == "__main__":
    main()
