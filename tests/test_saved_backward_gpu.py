"""GPU: a product's gradients from an operand and values before the activation that were
kept in 8 bits. Against 64-bit forms of the values that the 8 bits hold: the operand is made
again in fp32 (2e-6 (1 + |x|) for an activation, ops_util.py) and rounded once, D as in
linear_backward, and the products' sums are bounded as there."""
import pytest
import torch

from dense_gemm_gb300 import GemmError, linear_backward, quantize_rows, sync_status
from gpu_util import require_gpu
from ops_util import act, assert_close, rounding, strided, sum_error

pytestmark = pytest.mark.gpu
F16, BF16, F32, I8, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
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


def ints(g, *shape, dtype, hi=2):
    return torch.randint(-hi, hi + 1, shape, generator=g, device="cuda").to(F32).to(dtype)


def place(x, ld=None, offset=0):
    """8-bit x [r, c] with rows ld apart, offset bytes into a buffer of 127s (NaN in e4m3)."""
    r, c = x.shape
    ld = c if ld is None else ld
    buf = torch.full((offset + max(0, r - 1) * ld + c + 3,), 127, dtype=torch.uint8, device="cuda")
    v = buf.as_strided((r, c), (ld, 1), offset)
    v.copy_(x.view(torch.uint8))
    return v.view(x.dtype) if offset == 0 and ld == c else buf.view(x.dtype).as_strided((r, c), (ld, 1), offset)


SIZES = [(1, 64, 128), (3, 65, 33), (257, 1000, 513), (300, 264, 520), (1000, 72, 300), (40, 8, 1001)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("kept", [E4M3, I8])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("w_t", [False, True])
def test_integers_are_exact(size, kept, dtype, w_t):
    M, N, K = size
    g = gen(N)
    A, P = ints(g, M, K, dtype=kept), ints(g, M, N, dtype=kept)
    B, G = ints(g, K, N, dtype=dtype), ints(g, M, N, dtype=dtype)
    sa, sp = 2.0 ** torch.randint(-1, 2, (M,), generator=g, device="cuda").float(), 2.0 ** torch.randint(-1, 2, (M,), generator=g, device="cuda").float()
    W = strided(B, transposed=True) if w_t else B
    Ad, Pd = A.double() * sa.double()[:, None], P.double() * sp.double()[:, None]
    for act_a, activation in (("none", "relu"), ("relu", "none"), ("relu", "relu")):
        dA, dB, db = linear_backward(G, A, W, scale_a=sa, activation_a=act_a, pre=P, scale_pre=sp, activation=activation, need_bias=True, grad_dtype=F32)
        D = G.double() * (Pd > 0) if activation == "relu" else G.double()
        X = Ad.clamp_min(0) if act_a == "relu" else Ad
        assert torch.equal(dA.double(), D @ B.double().t())
        assert torch.equal(dB.double(), X.t() @ D)
        assert torch.equal(db.double(), D.sum(0))


@pytest.mark.parametrize("offset,pad", [(0, 8), (0, 16), (1, 0), (4, 4), (3, 5), (7, 2)])
@pytest.mark.parametrize("kept", [E4M3, I8])
def test_any_place_in_memory(offset, pad, kept):
    for M, N, K in ((9, 129, 200), (70, 264, 513), (33, 256, 640)):
        g = gen(offset + pad)
        A, P = ints(g, M, K, dtype=kept), ints(g, M, N, dtype=kept)
        B, G = ints(g, K, N, dtype=F16), ints(g, M, N, dtype=F16)
        one = torch.ones(M, device="cuda")
        want = linear_backward(G, A.to(F16), B, pre=P.to(F16), activation="relu", need_bias=True)
        got = linear_backward(strided(G, N + pad, offset), place(A, K + pad, offset), strided(B, N + pad, offset), scale_a=one,
                              pre=place(P, N + pad, 2 * offset), scale_pre=one, activation="relu", need_bias=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("act_a,activation", [("gelu", "none"), ("silu", "none"), ("gelu_tanh", "silu"), ("none", "gelu"), ("none", "gelu_tanh"),
                                              ("none", "silu"), ("relu", "gelu")])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [(5, 72, 130), (257, 1000, 513), (640, 512, 256)])
def test_random_gradients(act_a, activation, dtype, size):
    M, N, K = size
    g = gen(K)
    A, sa = quantize_rows(normal(g, M, K, scale=2))
    P, sp = quantize_rows(normal(g, M, N, scale=2), I8)
    B, G = normal(g, K, N, dtype=dtype, scale=K ** -0.5), normal(g, M, N, dtype=dtype)
    dA, dB, db = linear_backward(G, A, B, scale_a=sa, activation_a=act_a, pre=P, scale_pre=sp, activation=activation, need_bias=True)
    assert dA.dtype == dB.dtype == dtype and db.dtype == F32
    kept = A.double() * sa.double()[:, None]
    X = act(kept, act_a)
    eX = 1.13 * 2.0 ** -24 * kept.abs() + (2e-6 * (1 + kept.abs()) if act_a not in ("none", "relu") else 0)
    eX = eX + rounding(X, dtype)
    x = (P.double() * sp.double()[:, None]).requires_grad_()
    (slope,) = torch.autograd.grad(act(x, activation).sum(), x)
    x = x.detach()
    # the slope's own evaluation (4e-6 with the kept value's one rounding), then D's one rounding for the products
    eD = 5e-6 * G.double().abs() * (1 + x.abs()) if activation != "none" else torch.zeros_like(x)
    D = G.double() * slope
    eR = eD + rounding(D, dtype)
    assert_close(db, D.sum(0), eD.sum(0) + (M + 2) * 2.0 ** -24 * D.abs().sum(0), "dbias")
    Bd = B.double()
    assert_close(dA, D @ Bd.t(), eR @ Bd.abs().t() + sum_error(D, Bd.t()), "dA")
    assert_close(dB, X.t() @ D, X.abs().t() @ eR + eX.t() @ (D.abs() + eR) + sum_error(X.t(), D), "dB")


def test_either_may_be_kept_in_16_bits():
    g = gen(1)
    M, N, K = 50, 136, 72
    A, P, B, G = ints(g, M, K, dtype=BF16), ints(g, M, N, dtype=BF16), ints(g, K, N, dtype=BF16), ints(g, M, N, dtype=BF16)
    one = torch.ones(M, device="cuda")
    want = linear_backward(G, A, B, pre=P, activation="gelu", need_bias=True)
    for args in (dict(A=A.to(I8), scale_a=one, pre=P), dict(A=A, pre=P.to(E4M3), scale_pre=one), dict(A=A.to(E4M3), scale_a=one, pre=P.to(I8), scale_pre=one)):
        got = linear_backward(G, args.pop("A"), B, activation="gelu", need_bias=True, **args)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_that_are_not_needed_and_empty_sizes():
    g = gen(2)
    A, B, G, P = ints(g, 8, 16, dtype=E4M3), ints(g, 16, 24, dtype=F16), ints(g, 8, 24, dtype=F16), ints(g, 8, 24, dtype=I8)
    one = torch.ones(8, device="cuda")
    full = linear_backward(G, A, B, scale_a=one, pre=P, scale_pre=one, activation="relu", need_bias=True)
    for need in range(8):
        na, nb, nc = bool(need & 1), bool(need & 2), bool(need & 4)
        got = linear_backward(G, A, B, scale_a=one, pre=P, scale_pre=one, activation="relu", need_a=na, need_b=nb, need_bias=nc)
        for want, a, n in zip(full, got, (na, nb, nc)):
            assert torch.equal(a, want) if n else a is None
    got = linear_backward(G[:0], A[:0], B, scale_a=one[:0], pre=P[:0], scale_pre=one[:0], activation="relu", need_bias=True)
    assert got[0].shape == (0, 16) and (got[1] == 0).all() and (got[2] == 0).all()
    got = linear_backward(G, A[:, :0], B[:0], scale_a=one, need_bias=True)
    assert got[0].shape == (8, 0) and got[1].shape == (0, 24) and torch.equal(got[2], G.float().sum(0))


def test_a_scale_that_is_nan_reaches_the_gradients():
    g = gen(3)
    A, B, G = ints(g, 8, 16, dtype=I8), ints(g, 16, 24, dtype=F16), ints(g, 8, 24, dtype=F16)
    s = torch.ones(8, device="cuda")
    s[3] = float("nan")
    dA, dB, _ = linear_backward(G, A, B, scale_a=s)
    assert dB.isnan().all() and not dA.isnan().any()
    dA, dB, db = linear_backward(G, A, B, scale_a=torch.ones(8, device="cuda"), pre=ints(g, 8, 24, dtype=I8), scale_pre=s, activation="gelu", need_bias=True)
    assert dA[3].isnan().all() and not dA[2].isnan().any() and db.isnan().all()


def test_streams_workspaces_graphs_and_refusals():
    g = gen(4)
    M, N, K = 60, 129, 65
    A, B, G, P = ints(g, M, K, dtype=E4M3), ints(g, K, N, dtype=F16), ints(g, M, N, dtype=F16), ints(g, M, N, dtype=E4M3)
    one = torch.ones(M, device="cuda")
    args = dict(scale_a=one, activation_a="relu", pre=P, scale_pre=one, activation="relu", need_bias=True)
    want = linear_backward(G, A, B, **args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = linear_backward(G, A, B, stream=s, **args)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(linear_backward(G, A, B, workspace=ws, **args), want))
    graph, X = torch.cuda.CUDAGraph(), G.clone()
    with torch.cuda.graph(graph):
        got = linear_backward(X, A, B, **args)
    X.copy_(G.flip(0))
    graph.replay()
    X.copy_(G)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad, err in [(lambda: linear_backward(G, A, B), TypeError), (lambda: linear_backward(G, A, B, scale_a=one[:5]), ValueError),
                     (lambda: linear_backward(G, A, B, scale_a=one.half()), TypeError),
                     (lambda: linear_backward(G, A.to(F16), B, scale_a=one), ValueError),
                     (lambda: linear_backward(G, A.to(F16), B, activation_a="gelu"), ValueError),
                     (lambda: linear_backward(G, A, B, scale_a=one, pre=P, activation="gelu"), ValueError),
                     (lambda: linear_backward(G, A, B, scale_a=one, pre=P.to(F16), scale_pre=one, activation="gelu"), ValueError),
                     (lambda: linear_backward(G, A, B, scale_a=one, activation="gelu"), ValueError),
                     (lambda: linear_backward(G, A, B.float(), scale_a=one), TypeError),
                     (lambda: linear_backward(G.to(BF16), A, B, scale_a=one), ValueError),
                     (lambda: linear_backward(G, A, B, scale_a=one, activation_a="tanh"), ValueError),
                     (lambda: linear_backward(G, A.cpu(), B, scale_a=one), ValueError)]:
        with pytest.raises(err):
            bad()
    for bad in (lambda: linear_backward(G, strided(A.float().to(E4M3), transposed=True), B, scale_a=one),
                lambda: linear_backward(G, A, B, scale_a=one, workspace=ws[:128])):
        with pytest.raises(GemmError):
            bad()
