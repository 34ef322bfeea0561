"""GPU: a tensor that a call writes (out, h_out, pre) counts as changed for autograd: a graph that
saved its old values for its backward pass refuses to run, as after any operation in place. A refused call
changes nothing."""
import pytest
import torch

from dense_gemm_gb300 import (GemmError, layer_norm, layer_norm_backward, linear, quantize_rows, rms_norm, rms_norm_backward, sync_status)
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F16, I8 = torch.float16, torch.int8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def half(*shape):
    return torch.randn(*shape, device="cuda").half()


W = 64
CALLS = {
    "linear out": lambda t: linear(half(8, 32), half(32, W), out=t),
    "linear pre": lambda t: linear(half(8, 32), half(32, W), activation="gelu", pre=t),
    "linear residual as out": lambda t: linear(half(8, 32), half(32, W), residual=t, out=t),
    "rms_norm out": lambda t: rms_norm(half(8, W), half(W), out=t),
    "rms_norm h_out": lambda t: rms_norm(t, half(W), residual=half(8, W), h_out=t),
    "rms_norm_backward": lambda t: rms_norm_backward(t, half(8, W), half(W), torch.ones(8, device="cuda"), out=t),
    "layer_norm out": lambda t: layer_norm(half(8, W), half(W), out=t),
    "layer_norm h_out": lambda t: layer_norm(half(8, W), half(W), residual=t, h_out=t),
    "layer_norm_backward": lambda t: layer_norm_backward(half(8, W), half(8, W), half(W), *torch.ones(2, 8, device="cuda"), grad_h=t, out=t),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_graph_that_saved_the_old_values_refuses(name):
    leaf = half(8, W).requires_grad_()
    saved = leaf * 1
    loss = saved.square().sum()
    CALLS[name](saved.detach())
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.backward()


def test_eight_bit_outputs_count_too():
    q = torch.empty(8, W, dtype=I8, device="cuda")
    before = q._version
    quantize_rows(half(8, W), out=q)
    assert q._version == before + 1


def test_inputs_and_refused_calls_change_nothing():
    x, w, out = half(8, W), half(W), half(8, W)
    versions = [t._version for t in (x, w, out)]
    layer_norm(x, w)
    linear(x, half(W, W), residual=x)
    with pytest.raises(GemmError):
        layer_norm(x, w, out=out, eps=-1.0)
    with pytest.raises(GemmError):
        rms_norm(x, w, out=out, eps=-1.0)
    assert [t._version for t in (x, w, out)] == versions


def test_inference_tensors_are_written_as_before():
    with torch.inference_mode():
        x, out = half(8, W), half(8, W)
        layer_norm(x, half(W), out=out)
    want = layer_norm(x, w := half(W)).y
    assert layer_norm(x, w, out=out).y is out and torch.equal(out, want)
