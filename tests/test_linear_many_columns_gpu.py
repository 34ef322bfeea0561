"""GPU: products whose columns reach the largest size (2^31 - 1), where the last
tile is cut and its place plus a tile's width no longer fits 32 bits."""
import pytest
import torch

from dense_gemm_gb300 import linear, sync_status
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


@pytest.mark.parametrize("kernel", ["split", "pair"])
@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 128])
def test_the_last_column(kernel, N):
    """One row, K = 1, so that C is B times 2 exactly; C's row is followed by NaN."""
    B = torch.empty(1, N, device="cuda", dtype=BF16)
    B.view(torch.int16).random_(0x3000, 0x3f80)  # normal values between 4e-10 and 1
    buf = torch.full((2 ** 31 + 256,), float("nan"), device="cuda", dtype=BF16)
    out = buf.as_strided((1, N), (2 ** 31, 1))
    linear(torch.full((1, 1), 2.0, device="cuda", dtype=BF16), B, out=out, kernel=kernel)
    assert bool(buf[N:].isnan().all())
    for at in range(0, N, 1 << 28):
        assert torch.equal(out[0, at:at + (1 << 28)], B[0, at:at + (1 << 28)] * 2), at
