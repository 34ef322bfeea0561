"""GPU: every combination of residual, pre and bias in the product's epilogue, short
and long sums, one and several tiles per program, rows with and without 16-byte
boundaries; integers, so exact."""
import itertools

import pytest
import torch

from dense_gemm_gb300 import linear, sync_status
from gpu_util import require_gpu
from ops_util import outside_untouched, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def ints(g, *shape, dtype, hi=2):
    return torch.randint(-hi, hi + 1, shape, generator=g, device="cuda").float().to(dtype)


@pytest.mark.parametrize("kernel", ["pair", "split", "auto"])
@pytest.mark.parametrize("size", [(300, 264, 72), (130, 520, 2112), (2600, 2312, 64), (1100, 2304, 4224)])
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, F32), (E4M3, F16)])
@pytest.mark.parametrize("with_r,with_pre,gap", list(itertools.product([False, True], [False, True], [0, 3])))
def test_parts_of_the_epilogue(kernel, size, dtype, out_dtype, with_r, with_pre, gap):
    M, N, K = size
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    # a quarter of the products is not zero, so that 16-bit outputs hold every sum exactly (|sum| < 2048)
    A = ints(g, M, K, dtype=F32, hi=1) * (torch.rand(M, K, generator=g, device="cuda") < 0.25)
    B = ints(g, K, N, dtype=F32, hi=1)
    A, B = A.to(dtype), B.t().contiguous().to(dtype).t()
    bias, R = ints(g, N, dtype=F32), ints(g, M, N, dtype=out_dtype, hi=60)
    kw = dict(scale_a=torch.ones(M, device="cuda"), scale_b=torch.full((N,), 2.0, device="cuda")) if dtype == E4M3 else {}
    # the product of small integers is exact in fp32 in any order
    x = A.float().double() @ B.float().double() * (2 if dtype == E4M3 else 1) + bias.double()
    want = torch.where(x < 0, torch.zeros_like(x), x) + (R.double() if with_r else 0)
    place = lambda t: strided(t, N + gap, gap)
    for own in (False, True):  # the residual in C's place
        if own and not with_r:
            continue
        r = place(R) if with_r else None
        out = r if own else place(torch.zeros_like(R))
        pre = place(torch.zeros_like(R)) if with_pre else None
        linear(A, B, bias, activation="relu", residual=r, out=out, pre=pre, kernel=kernel, **kw)
        assert torch.equal(out.double(), want)
        if with_pre:
            assert torch.equal(pre.double(), x)
        if gap:
            assert outside_untouched(out) and (pre is None or outside_untouched(pre))
