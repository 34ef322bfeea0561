"""GPU: the product with its epilogue (linear) and its gradients against plain
64-bit forms; integer-valued inputs bit-exact."""
import itertools

import pytest
import torch

from dense_gemm_gb300 import GemmError, linear, linear_backward, sync_status
from gpu_util import require_gpu
from ops_util import act, assert_close, linear_ref, outside_untouched, rounding, strided, sum_error

pytestmark = pytest.mark.gpu

F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
KERNELS = ["pair", "split"]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def ints(g, *shape, dtype, hi=4):
    return torch.randint(-hi, hi + 1, shape, generator=g, device="cuda").to(F32).to(dtype)


# ------------------------------------------------------------------ exact: every size, type and layout

SIZES = [(1, 1, 1), (1, 128, 64), (2, 129, 65), (16, 256, 128), (17, 384, 200), (33, 1000, 72), (64, 130, 1024),
         (65, 257, 136), (130, 40, 520), (200, 300, 136), (257, 513, 72), (300, 600, 1000), (513, 512, 8)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32), (E4M3, BF16), (E4M3, F16),
                                             (E4M3, F32)])
def test_integers_are_exact(kernel, size, dtype, out_dtype):
    M, N, K = size
    g = gen(M + N + K)
    A, B = ints(g, M, K, dtype=dtype, hi=2), ints(g, N, K, dtype=dtype, hi=2).t()
    bias, res = ints(g, N, dtype=out_dtype, hi=8), ints(g, M, N, dtype=out_dtype, hi=8)
    sc = {}
    if dtype == E4M3:  # powers of two: exact
        sc = dict(scale_a=torch.exp2(torch.randint(-2, 3, (M,), generator=g, device="cuda").float()),
                  scale_b=torch.exp2(torch.randint(-2, 3, (N,), generator=g, device="cuda").float()))
    got, pre = linear(A, B, bias, activation="relu", residual=res, out_dtype=out_dtype, return_pre=True, kernel=kernel, **sc)
    c, x, _, _ = linear_ref(A.float(), B.float(), bias, "relu", res, **sc)
    assert torch.equal(got, c.to(out_dtype)) and torch.equal(pre, x.to(out_dtype))
    got = linear(A, B, residual=res, out_dtype=out_dtype, kernel=kernel, **sc)
    assert torch.equal(got, linear_ref(A.float(), B.float(), None, "none", res, **sc)[0].to(out_dtype))
    got = linear(A, B, out_dtype=out_dtype, kernel=kernel, **sc)
    assert torch.equal(got, linear_ref(A.float(), B.float(), **sc)[0].to(out_dtype))


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("a_t,b_t", list(itertools.product([False, True], repeat=2)))
@pytest.mark.parametrize("size", [(5, 200, 136), (100, 264, 256), (300, 520, 328)])
def test_operand_orders_are_exact(kernel, a_t, b_t, size):
    M, N, K = size
    g = gen(M + 2 * a_t + b_t)
    A, B = ints(g, M, K, dtype=F16), ints(g, K, N, dtype=F16)
    ref = (A.double() @ B.double()).to(F32)
    got = linear(strided(A, transposed=a_t), strided(B, transposed=b_t), out_dtype=F32, kernel=kernel)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [F16, E4M3])
@pytest.mark.parametrize("pads", [(8, 16, 0), (1, 3, 5), (7, 0, 1), (0, 8, 3)])
@pytest.mark.parametrize("size", [(3, 130, 257), (70, 300, 129), (300, 261, 72)])
def test_strides_offsets_and_untouched_gaps(kernel, dtype, pads, size):
    M, N, K = size
    pa, pb, off = pads
    g = gen(M + pa)
    A, B = ints(g, M, K, dtype=dtype, hi=2), ints(g, N, K, dtype=dtype, hi=2)
    bias, res = ints(g, N, dtype=F32, hi=9), ints(g, M, N, dtype=F16, hi=9)
    sc = dict(scale_a=torch.ones(M, device="cuda"), scale_b=torch.ones(N, device="cuda")) if dtype == E4M3 else {}
    out = strided(torch.zeros(M, N, dtype=F16, device="cuda"), N + pb, off)
    pre = strided(torch.zeros(M, N, dtype=F16, device="cuda"), N + pa, 2 * off)
    linear(strided(A, K + pa, off), strided(B, K + pb, off).t(), bias, residual=strided(res, N + pa, off), out=out, pre=pre,
           kernel=kernel, **sc)
    c, x, _, _ = linear_ref(A.float(), B.float().t(), bias, "none", res)
    assert torch.equal(out, c.to(F16)) and torch.equal(pre, x.to(F16))
    assert outside_untouched(out) and outside_untouched(pre)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("size", [(40, 256, 192), (600, 776, 192), (1100, 2304, 72)])
def test_residual_in_place(kernel, dtype, size):
    M, N, K = size
    g = gen(5)
    A, B, res = ints(g, M, K, dtype=F16), ints(g, K, N, dtype=F16), ints(g, M, N, dtype=dtype, hi=8)
    ref = linear_ref(A, B, None, "none", res)[0].to(dtype)
    assert torch.equal(linear(A, B, residual=res, out=res, kernel=kernel), ref)


@pytest.mark.parametrize("split_k", [64, 256, 512, 1024, 2048, 8192])
def test_cluster_sums_are_exact(split_k):
    """The K splits a cluster takes grow with K; every one sums to the same integers."""
    for M, N in [(1, 128), (3, 260), (48, 512), (130, 256)]:
        g = gen(split_k + M)
        A, B = ints(g, M, split_k, dtype=BF16, hi=2), ints(g, split_k, N, dtype=BF16, hi=2)
        assert torch.equal(linear(A, B, out_dtype=F32, kernel="split"), (A.double() @ B.double()).float())


def test_many_tiles_per_program_are_exact():
    """More tiles than CTA pairs: accumulators, buffers and residual fetches are reused."""
    M, N, K = 4000, 5000, 136
    g = gen(9)
    A, B, res = ints(g, M, K, dtype=F16, hi=2), ints(g, K, N, dtype=F16, hi=2), ints(g, M, N, dtype=F16, hi=8)
    bias = ints(g, N, dtype=F16, hi=8)
    for kernel in KERNELS:
        got, pre = linear(A, B, bias, activation="relu", residual=res, return_pre=True, kernel=kernel)
        c, x, _, _ = linear_ref(A, B, bias, "relu", res)
        assert torch.equal(got, c.to(F16)) and torch.equal(pre, x.to(F16))
        assert torch.equal(linear(A, B, bias, residual=res, kernel=kernel), (x + res.double()).to(F16))


# ------------------------------------------------------------------ random values, within the derived bound

@pytest.mark.parametrize("kernel", KERNELS + ["auto"])
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F16), (BF16, BF16), (BF16, F32), (E4M3, BF16)])
@pytest.mark.parametrize("size", [(4, 520, 264), (300, 390, 1000)])
def test_random_values(kernel, activation, dtype, out_dtype, size):
    M, N, K = size
    g = gen(M)
    sc = {}
    if dtype == E4M3:
        A, B = normal(g, M, K, scale=30).to(E4M3), normal(g, N, K, scale=30).to(E4M3).t()
        sc = dict(scale_a=torch.rand(M, generator=g, device="cuda") * 0.02 + 0.01,
                  scale_b=torch.rand(N, generator=g, device="cuda") * 0.002 + 0.001)
    else:
        A, B = normal(g, M, K, dtype=dtype), normal(g, K, N, dtype=dtype, scale=K ** -0.5)
    bias, res = normal(g, N), normal(g, M, N, dtype=out_dtype)
    got, pre = linear(A, B, bias, activation=activation, residual=res, out_dtype=out_dtype, return_pre=True,
                      kernel=kernel, **sc)
    c, x, ec, ex = linear_ref(A.float(), B.float(), bias, activation, res, **sc)
    assert_close(got, c, ec, "C")
    assert_close(pre, x, ex, "pre")


def test_same_call_twice_is_bit_identical():
    g = gen(3)
    for M, N, K in [(1, 4096, 4096), (48, 1000, 4096), (1000, 1000, 1000)]:
        A, B = normal(g, M, K, dtype=BF16), normal(g, K, N, dtype=BF16)
        assert torch.equal(linear(A, B), linear(A, B))


def test_nan_infinity_and_extremes():
    g = gen(4)
    for kernel, M in [("pair", 300), ("split", 5)]:
        A, B = ints(g, M, 64, dtype=BF16), ints(g, 64, 256, dtype=BF16)
        A[1, 3] = float("nan")
        A[2, 5] = float("inf")
        B[5, :] = 1.0
        got = linear(A, B, activation="relu", kernel=kernel)
        assert got[1].isnan().all() and (got[2] == float("inf")).all()
        assert not got[0].isnan().any() and not got[3:].isnan().any()
        bias = torch.full((256,), -3e4, device="cuda")
        z = torch.zeros_like(A)
        assert (linear(z, B, bias, activation="silu", kernel=kernel) == 0).all()
        assert (linear(z, B, -bias, activation="gelu_tanh", out_dtype=F32, kernel=kernel) == 3e4).all()
        assert (linear(z, B, bias, activation="gelu", out_dtype=F32, kernel=kernel).abs() == 0).all()


def test_empty_sizes():
    e = lambda *s: torch.zeros(*s, dtype=F16, device="cuda")  # noqa: E731
    assert linear(e(0, 8), e(8, 16)).shape == (0, 16)
    assert linear(e(4, 8), e(8, 0)).shape == (4, 0)
    bias, res = torch.arange(16, device="cuda").half() - 8, torch.ones(4, 16, device="cuda").half()
    got, pre = linear(e(4, 0), e(0, 16), bias, activation="relu", residual=res, return_pre=True)
    assert torch.equal(got, bias.clamp_min(0) + res) and torch.equal(pre, bias.expand(4, 16))
    dA, dB, db = linear_backward(e(0, 16), e(0, 8), e(8, 16), need_bias=True)
    assert dA.shape == (0, 8) and (dB == 0).all() and (db == 0).all()
    dA, dB, db = linear_backward(res, e(4, 0), e(0, 16), need_bias=True)
    assert dA.shape == (4, 0) and dB.shape == (0, 16) and torch.equal(db, torch.full((16,), 4.0, device="cuda"))


# ------------------------------------------------------------------ gradients

@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("size", [(1, 64, 128), (3, 65, 33), (257, 1000, 513), (300, 264, 520), (1000, 72, 300)])
@pytest.mark.parametrize("x_t,w_t", [(False, False), (False, True), (True, True)])
@pytest.mark.parametrize("activation", ["none", "relu"])
def test_integer_gradients_are_exact(kernel, size, x_t, w_t, activation):
    M, N, K = size
    g = gen(N)
    A, B, G = ints(g, M, K, dtype=F16, hi=2), ints(g, K, N, dtype=F16, hi=2), ints(g, M, N, dtype=F16, hi=2)
    P = ints(g, M, N, dtype=F16, hi=2) if activation == "relu" else None
    W = strided(B, transposed=True) if w_t else B
    X = strided(A, transposed=True) if x_t else A
    dA, dB, db = linear_backward(G, X, W, pre=P, activation=activation, need_bias=True, grad_dtype=F32, kernel=kernel)
    D = G.double() if P is None else G.double() * (P > 0)
    assert torch.equal(dA, (D @ B.double().t()).float())
    assert torch.equal(dB, (A.double().t() @ D).float())
    assert torch.equal(db, D.sum(0).float())


@pytest.mark.parametrize("activation", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [(5, 72, 130), (257, 1000, 513), (640, 512, 256)])
def test_random_gradients(activation, dtype, size):
    M, N, K = size
    g = gen(K)
    A, B = normal(g, M, K, dtype=dtype), normal(g, K, N, dtype=dtype, scale=K ** -0.5)
    G, P = normal(g, M, N, dtype=dtype), normal(g, M, N, dtype=dtype, scale=2)
    dA, dB, db = linear_backward(G, A, B, pre=P, activation=activation, need_bias=True)
    x = P.double().requires_grad_()
    (slope,) = torch.autograd.grad(act(x, activation).sum(), x)
    D = G.double() * slope
    # the slope's own evaluation (at most 4e-6), then D's one rounding for the products
    eD = 4e-6 * G.double().abs() * (1 + P.double().abs())
    eR = eD + rounding(D, dtype)
    assert_close(db, D.sum(0), eD.sum(0) + (M + 2) * 2.0 ** -24 * D.abs().sum(0), "dbias")
    Ad, Bd = A.double(), B.double()
    assert_close(dA, D @ Bd.t(), eR @ Bd.abs().t() + sum_error(D, Bd.t()), "dA")
    assert_close(dB, Ad.t() @ D, Ad.abs().t() @ eR + sum_error(Ad.t(), D), "dB")


@pytest.mark.parametrize("activation", ["none", "gelu", "gelu_tanh", "silu"])
def test_gradient_against_differences(activation):
    """d/dt sum(R * linear(A + t dA, ...)) by central differences of the forward
    kernel's fp32 output. With step t the third derivative's term is below t^2
    and the fp32 values' error, about 1e-6 of sums of magnitude 1, is divided by
    2t: t = 2^-5 leaves 1e-3 + 1e-4 of the gradient's scale; 16-bit gradients
    add 2^-8."""
    M, N, K = 24, 40, 64
    g = gen(8)
    A, B, bias, R = (normal(g, M, K, dtype=BF16), normal(g, K, N, dtype=BF16, scale=K ** -0.5), normal(g, N),
                     normal(g, M, N, dtype=BF16))
    # directions of +-t/4 steps that keep A + t V exact in bf16 are not needed: the
    # perturbed inputs are rounded first and the difference uses what was rounded
    t = 2.0 ** -5
    _, pre = linear(A, B, bias, activation=activation, return_pre=True)
    dA, dB, db = linear_backward(R, A, B, pre=pre, activation=activation, need_bias=True)

    def loss(A_, B_, bias_):
        return float((linear(A_, B_, bias_, activation=activation, out_dtype=F32).double() * R.double()).sum())
    for which in range(3):
        base = [A, B, bias]
        V = normal(g, *base[which].shape)
        hi, lo = list(base), list(base)
        hi[which] = (base[which].float() + t * V).to(base[which].dtype)
        lo[which] = (base[which].float() - t * V).to(base[which].dtype)
        grad = (dA, dB, db)[which].double()
        step = hi[which].double() - lo[which].double()
        want = loss(*hi) - loss(*lo)
        got = float((grad * step).sum())
        scale = float((grad * step).square().sum().sqrt())
        # pre and D rounded to bf16 (2^-9 each, random over the terms), plus the terms above
        assert abs(got - want) <= 0.03 * scale + 2e-3 * float((grad * step).abs().sum()), (which, got, want, scale)


def test_gradients_that_are_not_needed_are_not_made():
    g = gen(2)
    A, B, G = ints(g, 8, 16, dtype=F16), ints(g, 16, 24, dtype=F16), ints(g, 8, 24, dtype=F16)
    dA, dB, db = linear_backward(G, A, B, need_a=False)
    assert dA is None and db is None and torch.equal(dB, (A.double().t() @ G.double()).half())
    dA, dB, db = linear_backward(G, A, B, need_a=False, need_b=False, need_bias=True)
    assert dA is None and dB is None and torch.equal(db, G.float().sum(0))


# ------------------------------------------------------------------ streams, workspaces, refusals

def test_other_stream_and_given_workspace():
    g = gen(6)
    A, B = ints(g, 70, 257, dtype=F16), ints(g, 257, 301, dtype=F16)
    ref = (A.double() @ B.double()).half()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = linear(A, B, stream=s)
    s.synchronize()
    assert torch.equal(got, ref)
    from dense_gemm_gb300 import linear_workspace_size
    need = linear_workspace_size(A, B)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(linear(A, B, workspace=ws), ref)
    with pytest.raises(GemmError) as e:
        linear(A, B, workspace=ws[: need - 1])
    assert e.value.status == 1


def test_captured_in_a_graph():
    g = gen(7)
    A, B, res = ints(g, 16, 512, dtype=BF16, hi=2), ints(g, 512, 256, dtype=BF16, hi=2), ints(g, 16, 256, dtype=BF16)
    out = torch.empty_like(res)
    linear(A, B, residual=res, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        linear(A, B, residual=res, out=out)
    A.copy_(ints(g, 16, 512, dtype=BF16, hi=2))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, linear_ref(A, B, None, "none", res)[0].to(BF16))


def test_refusals():
    z = lambda *s, t=F16: torch.zeros(*s, device="cuda").to(t)  # noqa: E731
    A, B = z(4, 8), z(8, 16)
    for bad, err in [(lambda: linear(A, z(9, 16)), ValueError), (lambda: linear(A, z(8, 16, t=BF16)), TypeError),
                     (lambda: linear(A.float(), B.float()), TypeError), (lambda: linear(A.cpu(), B.cpu()), ValueError),
                     (lambda: linear(A, B, activation="tanh"), ValueError), (lambda: linear(A, B, z(15)), ValueError),
                     (lambda: linear(A, B, z(16, t=BF16)), TypeError), (lambda: linear(A, B, residual=z(4, 15)), ValueError),
                     (lambda: linear(A, B, residual=z(4, 16, t=BF16), out_dtype=F16), ValueError),
                     (lambda: linear(A, B, scale_a=z(4, t=F32), scale_b=z(16, t=F32)), ValueError),
                     (lambda: linear(A.to(E4M3), B.to(E4M3)), ValueError),
                     (lambda: linear(A, B, out=z(4, 16, t=torch.float64)), TypeError),
                     (lambda: linear(A, B, kernel="both"), ValueError),
                     (lambda: linear_backward(z(4, 16), A, B, activation="gelu"), ValueError),
                     (lambda: linear_backward(z(4, 16, t=BF16), A, B), ValueError)]:
        with pytest.raises(err):
            bad()
    one = torch.ones(8, device="cuda")
    for bad in (lambda: linear(A[:, ::2], B[::2]) if A[:, ::2].stride(0) == 1 else linear(z(8, 16)[::2, ::2], z(8, 16)),
                lambda: linear(A, B, out=z(16, 4).t()), lambda: linear(A[:1].expand(4, 8), B),
                lambda: linear(A, B, residual=z(1, 16).expand(4, 16)),
                lambda: linear(z(4, 8).to(E4M3), z(8, 16).to(E4M3), scale_a=one[:4], scale_b=z(16, t=F32))):
        with pytest.raises(GemmError):  # layouts the kernels do not take
            bad()
