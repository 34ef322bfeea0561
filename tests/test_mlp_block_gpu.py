"""GPU: the feed-forward block of examples/mlp_block.py, which runs the norm, the
product and their gradients together, against the same block in 64 bits."""
import importlib.util
import os

import pytest
import torch

from gpu_util import require_gpu
from ops_util import act

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mlp():
    require_gpu()
    from dense_gemm_gb300 import build, sync_status
    build.build()
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    yield module
    assert sync_status() == 0


def inputs(tokens, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3)]


def plain(block, x, r):
    """The block in float64, on leaves of its own: (out, leaves in the order x, norm, w1, b1, w2, b2)."""
    x, r, norm, w1, b1, w2, b2 = (t.detach().double().requires_grad_() for t in
                                  (x, r, block.norm, block.w1, block.b1, block.w2, block.b2))
    h = x + r
    y = norm * h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    return act(y @ w1.t() + b1, block.activation) @ w2.t() + b2 + h, (x, r, norm, w1, b1, w2, b2)


def relative(got, ref):
    return float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())


# One rounding to bf16 is at most 2^-8 of the value, and at most 2^-8 / sqrt(3) of it
# on average (root mean square). No value passes through more than eight (y, pre, u,
# D, du, dy, h and its own), whose errors are independent and carried on with slopes
# near one: sqrt(8) 2^-8 / sqrt(3) = 1.6 * 2^-8 of a tensor's norm; 2^-6 is 2.4 times that.
NORM_BOUND = 2.0 ** -6


@pytest.mark.parametrize("tokens,width,hidden", [(1, 256, 512), (37, 264, 520), (130, 257, 515), (512, 512, 1024)])
@pytest.mark.parametrize("activation", ["gelu", "silu"])
def test_forward_and_gradients(mlp, tokens, width, hidden, activation):
    block = mlp.MlpBlock(width, hidden, activation, seed=3)
    x, r, grad = inputs(tokens, width, 4)
    x, r = x.requires_grad_(), r.requires_grad_()
    out = block(x, r)
    out.backward(grad)
    ref, leaves = plain(block, x, r)
    ref.backward(grad.double())
    assert relative(out, ref) <= NORM_BOUND
    got = (x.grad, r.grad, block.norm.grad, block.w1.grad, block.b1.grad, block.w2.grad, block.b2.grad)
    for name, g, leaf in zip(("x", "r", "norm", "w1", "b1", "w2", "b2"), got, leaves):
        assert g.shape == leaf.shape
        assert relative(g, leaf.grad) <= NORM_BOUND, name
    assert torch.equal(block.serve(x, r), out)


def test_training_lowers_the_loss(mlp):
    block = mlp.MlpBlock(256, 1024, seed=5)
    x, r, target = inputs(96, 256, 6)
    losses = mlp.train(block, x, r, target.float(), 30)
    assert losses[-1] < 0.9 * losses[0]


def test_eight_bits_and_single_tokens(mlp):
    block = mlp.MlpBlock(512, 1024, seed=7)
    low = mlp.EightBitBlock(block)
    x, r, _ = inputs(5, 512, 8)
    with torch.no_grad():
        ref = plain(block, x, r)[0]
        # two operands of 3 mantissa bits: 2^-4 each at most, so 2^-3 of the branch's norm
        branch = ref - (x.double() + r.double())
        assert float((low.serve(x, r).double() - ref).norm() / branch.norm()) <= 2.0 ** -3
    for serve in (block.serve, low.serve):
        graph, gx, gr, out = mlp.captured(serve, x[:1], r[:1])
        for i in range(5):  # other inputs through the same graph
            gx.copy_(x[i:i + 1])
            gr.copy_(r[i:i + 1])
            graph.replay()
            assert torch.equal(out, serve(x[i:i + 1], r[i:i + 1]))
