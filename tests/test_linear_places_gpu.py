"""GPU: gradients of the product whose G and pre lie at any place of a 16-byte
granule, each at its own, with NaN around their rows; integers, so exact."""
import itertools

import pytest
import torch

from dense_gemm_gb300 import linear_backward, sync_status
from gpu_util import require_gpu
from ops_util import strided

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def ints(seed, *shape, dtype, hi=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-hi, hi + 1, shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("size", [(1, 1, 1), (3, 7, 5), (17, 9, 64), (70, 257, 40), (33, 1001, 24), (200, 511, 72), (9, 2056, 16)])
@pytest.mark.parametrize("places", list(itertools.product([(0, 0), (1, 3)], [(0, 0), (3, 5), (8, 7)])))
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_from_any_place(size, places, dtype):
    M, N, K = size
    (ga, oa), (gp, op) = places
    G, P = ints(1, M, N, dtype=dtype), ints(2, M, N, dtype=dtype)
    A, B = ints(3, M, K, dtype=dtype), ints(4, K, N, dtype=dtype)
    g, pre = strided(G, N + ga, oa), strided(P, N + gp, op)
    D = torch.where(P.double() > 0, G.double(), torch.zeros((), device="cuda", dtype=torch.float64))
    for act, want in (("relu", D), ("none", G.double())):
        dA, dB, db = linear_backward(g, A, B, pre=pre if act == "relu" else None, activation=act, need_bias=True,
                                     grad_dtype=torch.float32)
        assert torch.equal(db.double(), want.sum(0)), act
        assert torch.equal(dA.double(), want @ B.double().t()), act
        assert torch.equal(dB.double(), A.double().t() @ want), act


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
def test_same_values_as_aligned(activation):
    """Where a row lies changes nothing: bit for bit the aligned call's D and sums."""
    M, N, K = 300, 1024, 64
    gen = torch.Generator(device="cuda").manual_seed(5)
    G, P, A, B = (torch.randn(*s, generator=gen, device="cuda").to(BF16) for s in ((M, N), (M, N), (M, K), (K, N)))
    want = linear_backward(G, A, B, pre=P, activation=activation, need_bias=True)
    got = linear_backward(strided(G, N + 1, 1), A, B, pre=strided(P, N + 3, 2), activation=activation, need_bias=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
