"""GPU: the norm's gradients written over one of their inputs. dx and dweight are
those of the same call with an output of its own, also where the rows are too
long for the kernels that keep them on chip and dx and dweight come from two
passes over the inputs."""
import pytest
import torch

from dense_gemm_gb300 import rms_norm_backward, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, outside_untouched, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def normal(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# (type, rows, width, offset of grad's and dx's first element, of h's, of grad_h's): rows
# in registers, through shared memory and in two passes; aligned, all at one place, at places of their own
CASES = [(F32, 70, 512, 0, 0, 0), (F32, 40, 4096, 0, 0, 0), (F32, 640, 5120, 0, 0, 0), (F32, 33, 7168, 0, 0, 0),
         (F32, 700, 8192, 0, 0, 0), (F32, 9, 9216, 0, 0, 0), (F32, 5, 16384, 0, 0, 0), (F32, 12, 5120, 1, 2, 3),
         (F16, 50, 4096, 0, 0, 0), (F16, 50, 4095, 3, 3, 3), (F16, 6, 16384, 0, 0, 0), (F16, 700, 16392, 0, 0, 0),
         (BF16, 50, 20000, 0, 0, 0), (BF16, 40, 9001, 1, 2, 3), (BF16, 640, 16001, 1, 2, 3), (BF16, 3, 16377, 5, 5, 5),
         (BF16, 1, 33000, 0, 0, 0)]


@pytest.mark.parametrize("through", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_gradients_over_an_input(case, through):
    dtype, rows, width, og, oh, od = case
    dy, h, w = normal(1, rows, width, dtype=dtype), normal(2, rows, width, dtype=dtype), normal(3, width, dtype=dtype)
    dh = normal(4, rows, width, dtype=dtype) if through else None
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    at = lambda t, offset: strided(t, width, offset)
    given = dict(h=at(h, oh), weight=w, rstd=rstd)
    apart = at(torch.zeros_like(dy), og)
    dx, dw = rms_norm_backward(at(dy, og), grad_h=None if dh is None else at(dh, od), out=apart, **given)
    assert dx is apart
    terms = dy.double() * h.double() * rstd.double()[:, None]
    # three factors' roundings, then one addition a row
    assert_close(dw, terms.sum(0), (rows + 8) * 2.0 ** -24 * terms.abs().sum(0), "dweight")
    own = at(dy, og)
    got, dw2 = rms_norm_backward(own, grad_h=None if dh is None else at(dh, od), out=own, **given)
    assert got is own and torch.equal(got, dx) and torch.equal(dw2, dw) and outside_untouched(own)
    if not through:
        return
    # over grad_h, from one place for all calls: the same kernels, so the same bits
    apart = at(torch.zeros_like(dy), od)
    dx, dw = rms_norm_backward(at(dy, og), grad_h=at(dh, od), out=apart, **given)
    own = at(dh, od)
    got, dw2 = rms_norm_backward(at(dy, og), grad_h=own, out=own, **given)
    assert torch.equal(got, dx) and torch.equal(dw2, dw) and outside_untouched(own)
