#!/usr/bin/env python3
"""A transformer's feed-forward block on the library's operators, trained and served.

    python examples/mlp_block.py [--width 4096] [--hidden 16384] [--tokens 2048] [--steps 20]

    h = x + r;  y = rms_norm(h);  u = gelu(y W1 + b1);  out = u W2 + b2 + h

Training runs each part and its gradients through one autograd function per
operator. Serving has two forms: 16-bit weights, and 8-bit weights for W1, whose
operand the norm writes in 8 bits with a scale per row. A single token's step is
captured in a CUDA graph. Data and weights are synthetic.
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_gemm_gb300 import linear, linear_backward, rms_norm, rms_norm_backward

E4M3_MAX = 448.0


class Norm(torch.autograd.Function):
    """(y, h) of x, the residual stream r and the weight."""

    @staticmethod
    def forward(ctx, x, r, weight):
        n = rms_norm(x, weight, residual=r, return_rstd=True)
        ctx.save_for_backward(n.h, weight, n.rstd)
        return n.y, n.h

    @staticmethod
    def backward(ctx, grad_y, grad_h):
        h, weight, rstd = ctx.saved_tensors
        dx, dweight = rms_norm_backward(grad_y.contiguous(), h, weight, rstd, grad_h=grad_h.contiguous())
        return dx, dx, dweight.to(weight.dtype)


class Linear(torch.autograd.Function):
    """act(a W^T + bias) + residual, W kept as [out, in]."""

    @staticmethod
    def forward(ctx, a, W, bias, activation, residual):
        ctx.activation, ctx.has_residual = activation, residual is not None
        if activation == "none":
            ctx.save_for_backward(a, W, None)
            return linear(a, W.t(), bias, residual=residual)
        out, pre = linear(a, W.t(), bias, activation=activation, residual=residual, return_pre=True)
        ctx.save_for_backward(a, W, pre)
        return out

    @staticmethod
    def backward(ctx, grad):
        a, W, pre = ctx.saved_tensors
        grad = grad.contiguous()
        da, dw, dbias = linear_backward(grad, a, W.t(), pre=pre, activation=ctx.activation, need_bias=True)
        return da, dw.t(), dbias, None, grad if ctx.has_residual else None


class MlpBlock(torch.nn.Module):
    def __init__(self, width, hidden, activation="gelu", dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(out, into):
            return torch.nn.Parameter((torch.randn(out, into, generator=g, device=device) * into ** -0.5).to(dtype))

        self.activation = activation
        self.norm = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        self.w1, self.b1 = weight(hidden, width), torch.nn.Parameter(torch.zeros(hidden, device=device))
        self.w2, self.b2 = weight(width, hidden), torch.nn.Parameter(torch.zeros(width, device=device))

    def forward(self, x, r):
        """The block's output (the next residual stream) for x [tokens, width] and r; differentiable."""
        y, h = Norm.apply(x, r, self.norm)
        u = Linear.apply(y, self.w1, self.b1, self.activation, None)
        return Linear.apply(u, self.w2, self.b2, "none", h)

    @torch.no_grad()
    def serve(self, x, r):
        """The same without what the gradients need."""
        n = rms_norm(x, self.norm, residual=r)
        u = linear(n.y, self.w1.t(), self.b1, activation=self.activation)
        return linear(u, self.w2.t(), self.b2, residual=n.h)


class EightBitBlock:
    """``MlpBlock.serve`` with W1 in 8-bit floats, a scale per output."""

    @torch.no_grad()
    def __init__(self, block):
        self.block = block
        w = block.w1.float()
        self.scale = (w.abs().amax(1) / E4M3_MAX).clamp(min=1e-12)
        self.w1 = (w / self.scale[:, None]).to(torch.float8_e4m3fn)

    @torch.no_grad()
    def serve(self, x, r):
        b = self.block
        n = rms_norm(x, b.norm, residual=r, out_dtype=torch.float8_e4m3fn)
        u = linear(n.y, self.w1.t(), b.b1, activation=b.activation, scale_a=n.scale, scale_b=self.scale,
                   out_dtype=x.dtype)
        return linear(u, b.w2.t(), b.b2, residual=n.h)


def captured(serve, x, r):
    """(graph, x, r, out): one call of ``serve`` as a CUDA graph on buffers of its own."""
    x, r = x.clone(), r.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve(x, r)  # first use sets the library up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = serve(x, r)
    return graph, x, r, out


def train(block, x, r, target, steps, change=1e-3):
    """Losses of ``steps`` steps towards ``target``, each along the gradient and
    changing every parameter tensor by ``change`` (root mean square)."""
    losses = []
    for _ in range(steps):
        block.zero_grad(set_to_none=True)
        loss = (block(x, r).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in block.parameters():
                g = p.grad.float()
                p.copy_(p - change * g / g.square().mean().sqrt().clamp(min=1e-20))
        losses.append(float(loss.detach()))
    return losses


def microseconds(graph, n=200):
    for _ in range(10):
        graph.replay()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        graph.replay()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) * 1e3 / n


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=16384)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    block = MlpBlock(a.width, a.hidden)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, target = (torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16() for _ in range(3))
    losses = train(block, x, r, target.float(), a.steps)
    print(f"trained {a.steps} steps on {a.tokens} tokens: loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    low = EightBitBlock(block)
    full, eight = block.serve(x, r).float(), low.serve(x, r).float()
    print(f"8-bit W1: relative difference of the block's output {float((eight - full).norm() / full.norm()):.4f}")
    for name, serve in (("16-bit", block.serve), ("8-bit W1", low.serve)):
        graph = captured(serve, x[:1], r[:1])[0]
        print(f"{name}: {microseconds(graph):.1f} us for one token (weights may stay in L2)")


if __name__ == "__main__":
    main()
