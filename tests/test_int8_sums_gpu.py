"""GPU: products of 8-bit integers whose sums leave what fp32 holds exactly, or cancel after they did:
within (K + 16) 2^-23 of the sum of magnitudes (ops_util.sum_error), in the form for few
tokens, the one whose tokens come as fp16 and the one that copies both operands. Scales that
are NaN, and C past 2^31 elements."""
import pytest
import torch

from dense_gemm_gb300 import linear, sync_status
from gpu_util import require_gpu
from ops_util import sum_error

pytestmark = pytest.mark.gpu
F32, BF16, I8 = torch.float32, torch.bfloat16, torch.int8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(g, *shape, lo=-128, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(I8)


def product(A, W):
    one = torch.ones(max(A.shape[0], W.shape[0]), device="cuda")
    return linear(A, W.t(), scale_a=one[:A.shape[0]], scale_b=one[:W.shape[0]], out_dtype=F32)


def check(A, W):
    a, w = A.double(), W.double().t()
    got, want = product(A, W).double(), a @ w
    assert ((got - want).abs() <= sum_error(a, w)).all()
    return want


@pytest.mark.parametrize("M", [1, 33, 64, 100, 300, 1000])
@pytest.mark.parametrize("K", [1041, 4000, 16384])
def test_positive_values(M, K):
    """What a relu leaves: from K = 1041 on the largest values' sum is past 2^24."""
    g = gen(M + K)
    A, W = ints(g, M, K, lo=100), ints(g, 260, K, lo=100)
    assert check(A, W).min() > 2 ** 23
    A.fill_(127)
    W.fill_(127)
    assert check(A, W).min() > 2 ** 24


@pytest.mark.parametrize("M", [1, 33, 64, 100, 300, 1000])
@pytest.mark.parametrize("K", [2048, 4001, 16000])
def test_large_sums_that_cancel(M, K):
    """The first half of K adds up to more than 2^24, the second takes it away again but for a little."""
    g = gen(K)
    A, W = ints(g, M, K, lo=120), ints(g, 260, K, lo=110)
    half = K // 2
    A[:, half:2 * half] = A[:, :half]
    W[:, half:2 * half] = -W[:, :half]
    W[:, K - 1] = torch.arange(260, device="cuda").remainder(100).to(I8)
    want = check(A, W)
    if K > 4000:
        assert float((want.abs().max() / (A[:, :half].double() @ W[:, :half].double().t()).min())) < 0.02


@pytest.mark.parametrize("M", [1, 64, 100, 1000])
def test_exact_to_the_last_value_below(M):
    """K = 1024 of the largest magnitudes: 2^24, still a number of fp32."""
    A, W = torch.full((M, 1024), -128, dtype=I8, device="cuda"), torch.full((257, 1024), -128, dtype=I8, device="cuda")
    W[3] = 127
    want = A.double() @ W.double().t()
    assert torch.equal(product(A, W).double(), want) and want.max() == 2 ** 24


@pytest.mark.parametrize("M", [3, 64, 100, 1000])
def test_a_nan_scale_reaches_its_row_or_column_only(M):
    g = gen(M)
    K, N = 1024, 1100
    A, W = ints(g, M, K), ints(g, N, K)
    sa, sb = torch.rand(M, generator=g, device="cuda") + 0.5, torch.rand(N, generator=g, device="cuda") + 0.5
    want = linear(A, W.t(), scale_a=sa, scale_b=sb)
    sa[1], sb[7], sb[N - 1] = float("nan"), float("nan"), float("inf")
    got = linear(A, W.t(), scale_a=sa, scale_b=sb)
    assert got[1].isnan().all() and got[:, 7].isnan().all() and not got[:, N - 1].isfinite().any()
    rows, cols = torch.arange(M, device="cuda") != 1, torch.ones(N, dtype=torch.bool, device="cuda")
    cols[7] = cols[N - 1] = False
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])


@pytest.mark.parametrize("M,N,K", [(700, 3100000, 16), (66000, 33000, 48)])
def test_outputs_past_two_to_the_31(M, N, K):
    """Small whole numbers: exact in bf16."""
    g = gen(N)
    A, W = ints(g, M, K, lo=-2, hi=2), ints(g, N, K, lo=-2, hi=2)
    one = torch.ones(max(M, N), device="cuda")
    got = linear(A, W.t(), scale_a=one[:M], scale_b=one[:N])
    assert got.numel() > 2 ** 31
    for r0 in range(0, M, 8192):
        for c0 in (0, N // 2 - 300, N - 600):
            want = A[r0:r0 + 8192].float() @ W[c0:c0 + 600].float().t()
            assert torch.equal(got[r0:r0 + 8192, c0:c0 + 600].float(), want)
    for c0 in range(0, N, 1 << 18):
        want = A[M - 5:].float() @ W[c0:c0 + (1 << 18)].float().t()
        assert torch.equal(got[M - 5:, c0:c0 + (1 << 18)].float(), want)
