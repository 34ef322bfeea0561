"""GPU: the feed-forward block of examples/eight_bit_block.py, which runs layer norm, the
product, rows in 8 bits and the gradients from them together, against the same block in
64 bits."""
import importlib.util
import os

import pytest
import torch

from gpu_util import require_gpu
from ops_util import act

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    from dense_gemm_gb300 import build, sync_status
    build.build()
    spec = importlib.util.spec_from_file_location("eight_bit_block", os.path.join(ROOT, "examples", "eight_bit_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    assert sync_status() == 0


def inputs(tokens, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3)]


def plain(block, x, r):
    """The block in float64, on leaves of its own: (out, leaves in the order x, gain, shift, w1, b1, w2, b2)."""
    x, r, gain, shift, w1, b1, w2, b2 = (t.detach().double().requires_grad_() for t in
                                         (x, r, block.gain, block.shift, block.w1, block.b1, block.w2, block.b2))
    h = x + r
    c = h - h.mean(1, keepdim=True)
    y = gain * c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() + shift
    return act(y @ w1.t() + b1, "gelu") @ w2.t() + b2 + h, (x, r, gain, shift, w1, b1, w2, b2)


def relative(got, ref):
    return float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())


# Values in 16 bits as in test_mlp_block_gpu.py: 2^-6 of a tensor's norm. One rounding to e4m3
# is at most 2^-4 of the value, 2^-4 / sqrt(3) on average. A gradient of the block carries at
# most three of them (the operand kept; D, through gelu'; the operand made again, through
# gelu, whose relative slope p gelu'(p) / gelu(p) is at most 1.5 where gelu(p) is not small),
# independent of one another: sqrt(3) 1.5 2^-4 / sqrt(3) = 0.094; 2^-3 is 1.3 times that.
NORM_BOUND, KEPT_BOUND = 2.0 ** -6, 2.0 ** -3


@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (37, 264, 520), (130, 257, 515), (512, 512, 1024)])
def test_forward_and_gradients(example, tokens, width, hidden):
    block = example.EightBitBlock(width, hidden, seed=3)
    x, r, grad = inputs(tokens, width, 4)
    x, r = x.requires_grad_(), r.requires_grad_()
    out = block(x, r)
    out.backward(grad)
    ref, leaves = plain(block, x, r)
    ref.backward(grad.double())
    assert relative(out, ref) <= NORM_BOUND
    got = (x.grad, r.grad, block.gain.grad, block.shift.grad, block.w1.grad, block.b1.grad, block.w2.grad, block.b2.grad)
    for name, g, leaf in zip(("x", "r", "gain", "shift", "w1", "b1", "w2", "b2"), got, leaves):
        assert g.shape == leaf.shape
        assert relative(g, leaf.grad) <= (NORM_BOUND if name == "b2" else KEPT_BOUND), name
    assert torch.equal(block.serve(x, r), out)


def test_training_runs_and_single_tokens(example):
    """Weights and tokens in integers: a step is a / 127, so an operand is off by (a / 127) / sqrt(12)
    on average, a being some 4 deviations: 0.9 % of its norm; four operands 1.8 %, and 2^-4 is 3.4
    times that."""
    block = example.EightBitBlock(512, 1024, seed=7)
    x, r, target = inputs(5, 512, 8)
    losses = example.train(block, x, r, target.float(), 3)
    assert len(losses) == 3 and all(v == v for v in losses)
    low = example.IntegerBlock(block)
    with torch.no_grad():
        ref = plain(block, x, r)[0]
        branch = ref - (x.double() + r.double())
        assert float((low.serve(x, r).double() - ref).norm() / branch.norm()) <= 2.0 ** -4
    for serve in (block.serve, low.serve):
        graph, gx, gr, out = example.captured(serve, x[:1], r[:1])
        for i in range(5):  # other inputs through the same graph
            gx.copy_(x[i:i + 1])
            gr.copy_(r[i:i + 1])
            graph.replay()
            assert torch.equal(out, serve(x[i:i + 1], r[i:i + 1]))
