"""GPU: gradient calls of several sizes in a row that share one workspace, whose
kernels read what was written two launches earlier without waiting again: no
value of an earlier call, at the same address, may be taken for it."""
import pytest
import torch

from dense_gemm_gb300 import linear_backward, sync_status
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F16, F32 = torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


# operands copied (odd sizes) or not, column sums in one part or many, one or both products
SIZES = [(257, 1000, 513), (640, 520, 130), (64, 1000, 513), (1000, 257, 65), (7, 129, 33), (300, 264, 136)]


@pytest.mark.parametrize("activation", ["none", "relu"])
@pytest.mark.parametrize("both", [False, True])
def test_no_value_of_an_earlier_call(activation, both):
    g = torch.Generator(device="cuda").manual_seed(5)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(F16)
    ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    sets = [(M, N, K, ints(M, K), ints(K, N), [ints(M, N) for _ in range(3)], [ints(M, N) for _ in range(3)],
             torch.zeros(M, N, device="cuda", dtype=F16), torch.zeros(M, N, device="cuda", dtype=F16)) for M, N, K in SIZES]
    torch.cuda.synchronize()
    got = []
    for i in range(10 * len(sets)):
        M, N, K, A, B, grads, pres, G, P = sets[(i * 5) % len(sets)]
        k = i % 3
        G.copy_(grads[k])  # the kernel right before the call writes what it reads
        P.copy_(pres[(k + i // 3) % 3])
        got.append(((i * 5) % len(sets), k, (k + i // 3) % 3,
                    linear_backward(G, A, B, pre=P if activation != "none" else None, activation=activation, need_a=both,
                                    need_bias=True, grad_dtype=F32, workspace=ws)))
    torch.cuda.synchronize()
    for s, k, j, (dA, dB, db) in got:
        M, N, K, A, B, grads, pres, _, _ = sets[s]
        D = grads[k].double() * ((pres[j] > 0) if activation == "relu" else 1)
        assert torch.equal(db, D.sum(0).float()) and torch.equal(dB, (A.double().t() @ D).float())
        assert dA is None if not both else torch.equal(dA, (D @ B.double().t()).float())
