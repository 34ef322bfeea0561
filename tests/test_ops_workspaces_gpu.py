"""GPU: workspaces given by the caller. A tensor whose bytes are not all its own
(expanded, or with gaps) is refused before anything is launched."""
import pytest
import torch

from dense_gemm_gb300 import linear, linear_backward, linear_workspace_size, rms_norm_backward, sync_status
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def ints(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(F16)


A, B, G = (lambda: ints(1, 33, 65)), (lambda: ints(2, 65, 129)), (lambda: ints(3, 33, 129))
CALLS = {"linear": lambda ws: linear(A(), B(), workspace=ws),
         "linear_backward": lambda ws: linear_backward(G(), A(), B(), need_bias=True, workspace=ws)[1],
         "rms_norm_backward": lambda ws: rms_norm_backward(G(), G(), ints(4, 129), torch.ones(33, device="cuda"), workspace=ws)[1]}


@pytest.mark.parametrize("call", list(CALLS))
def test_a_workspace_has_bytes_of_its_own(call):
    n = 1 << 20
    assert linear_workspace_size(A(), B()) <= n  # it does need one: rows of 65 and 129 elements are copied
    want = CALLS[call](None)
    for good in (torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(256, n // 1024, device="cuda")):
        assert torch.equal(CALLS[call](good), want)
    backing = torch.empty(2 * n, dtype=torch.uint8, device="cuda")
    for bad in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), backing[::2], backing.view(2, n).t()):
        with pytest.raises(ValueError, match="contiguous"):
            CALLS[call](bad)
