"""GPU: products of 8-bit integers with scales for each token and channel. While the sum
of magnitudes stays below 2^24 the sums are exact, so with scales that are powers of two
the whole result is; beyond, the bound of an fp32 sum holds (ops_util.py)."""
import pytest
import torch

from dense_gemm_gb300 import GemmError, linear, linear_workspace_size, quantize_rows, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, linear_ref, outside_untouched, strided

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


def ints(g, *shape, lo=-128, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(I8)


def normal(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def place(x, ld=None, offset=0):
    """x [r, c] of int8 with rows ld apart, offset bytes into a buffer that is 85 elsewhere."""
    r, c = x.shape
    ld = c if ld is None else ld
    buf = torch.full((offset + max(0, r - 1) * ld + c + 3,), 85, dtype=I8, device="cuda")
    return buf.as_strided((r, c), (ld, 1), offset).copy_(x)


# K up to 1024 with |values| up to 128: below 2^24
SIZES = [(1, 1, 1), (1, 128, 128), (1, 257, 33), (3, 65, 7), (5, 1000, 1000), (16, 128, 1024), (17, 300, 513), (33, 4096, 256), (64, 129, 1000),
         (65, 130, 255), (128, 384, 640), (200, 520, 1000), (257, 1000, 513), (700, 72, 300), (600, 1000, 1000), (1000, 1024, 1024), (1030, 1100, 1024), (48, 16384, 512), (300, 3000, 1001),
         (65, 16000, 1000), (129, 8200, 840), (900, 1100, 1023)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("kernel", ["auto", "pair", "split"])
def test_exact_in_every_size(size, kernel):
    M, N, K = size
    g = gen(M + N + K)
    A, W = ints(g, M, K), ints(g, N, K)
    sa, sb = 2.0 ** torch.randint(-6, 3, (M,), generator=g, device="cuda").float(), 2.0 ** torch.randint(-6, 3, (N,), generator=g, device="cuda").float()
    want = (A.double() @ W.double().t()) * sa.double()[:, None] * sb.double()
    got = linear(A, W.t(), scale_a=sa, scale_b=sb, out_dtype=F32, kernel=kernel)
    assert torch.equal(got.double(), want)
    assert linear(A, W.t(), scale_a=sa, scale_b=sb).dtype == BF16


@pytest.mark.parametrize("value", [-128, 127])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_extreme_values(value, M):
    A, W = torch.full((M, 1000), value, dtype=I8, device="cuda"), torch.full((200, 1000), -128, dtype=I8, device="cuda")
    one = torch.ones(max(M, 200), device="cuda")
    assert (linear(A, W.t(), scale_a=one[:M], scale_b=one[:200], out_dtype=F32) == -128000 * value).all()


@pytest.mark.parametrize("offset,pad", [(0, 16), (0, 8), (8, 0), (1, 0), (3, 5), (4, 2), (15, 1)])
@pytest.mark.parametrize("size", [(1, 129, 200), (7, 300, 513), (40, 128, 1000), (130, 257, 640)])
def test_any_place_in_memory(offset, pad, size):
    M, N, K = size
    g = gen(offset + pad)
    A, W = ints(g, M, K), ints(g, N, K)
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    want = (A.double() @ W.double().t()).float()
    out = strided(torch.zeros(M, N, device="cuda"), N + 3, 1)
    got = linear(place(A, K + pad, offset), place(W, K + pad, 2 * offset).t(), scale_a=sa, scale_b=sb, out=out)
    assert torch.equal(got, want) and outside_untouched(out)


@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("out_dtype", [F16, BF16, F32])
@pytest.mark.parametrize("size", [(1, 520, 1500), (19, 333, 3000), (64, 1024, 2048), (300, 264, 4096)])
def test_the_whole_epilogue(activation, out_dtype, size):
    M, N, K = size
    g = gen(K)
    A, sa = quantize_rows(normal(g, M, K), I8)
    W, sb = quantize_rows(normal(g, N, K, scale=K ** -0.5), I8)
    bias, res = normal(g, N), normal(g, M, N, dtype=out_dtype)
    for b, r in ((bias, res), (bias.to(out_dtype), None), (None, res)):
        got, pre = linear(A, W.t(), b, activation=activation, residual=r, scale_a=sa, scale_b=sb, out_dtype=out_dtype, return_pre=True)
        c, x, ec, ex = linear_ref(A.float(), W.float().t(), b, activation, r, sa, sb)
        assert_close(got, c, ec, "C")
        assert_close(pre, x, ex, "pre")
        assert torch.equal(linear(A, W.t(), b, activation=activation, residual=r, scale_a=sa, scale_b=sb, out_dtype=out_dtype), got)


def test_sums_past_two_to_the_24():
    A = torch.full((3, 8192), 127, dtype=I8, device="cuda")
    W = torch.full((130, 8192), 127, dtype=I8, device="cuda")
    W[1] = -127
    one = torch.ones(130, device="cuda")
    got = linear(A, W.t(), scale_a=one[:3], scale_b=one, out_dtype=F32)
    c, _, e, _ = linear_ref(A.float(), W.float().t(), None, "none", None, one[:3], one)
    assert_close(got, c, e)


def test_empty_sizes_streams_workspaces_and_graphs():
    g = gen(5)
    z = lambda *s: torch.zeros(*s, dtype=I8, device="cuda")  # noqa: E731
    one = torch.ones(300, device="cuda")
    assert linear(z(0, 8), z(16, 8).t(), scale_a=one[:0], scale_b=one[:16]).shape == (0, 16)
    assert linear(z(4, 8), z(0, 8).t(), scale_a=one[:4], scale_b=one[:0]).shape == (4, 0)
    b = normal(g, 16)
    assert torch.equal(linear(z(4, 0), z(16, 0).t(), b, scale_a=one[:4], scale_b=one[:16], out_dtype=F32), b.expand(4, 16))
    for M in (3, 200):
        A, W = ints(g, M, 400), ints(g, 300, 400)
        want = (A.double() @ W.double().t()).float()
        args = dict(scale_a=one[:M], scale_b=one, out_dtype=F32)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = linear(A, W.t(), stream=s, **args)
        s.synchronize()
        assert torch.equal(got, want)
        need = linear_workspace_size(A, W.t())
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        assert torch.equal(linear(A, W.t(), workspace=ws, **args), want)
        if need:
            with pytest.raises(GemmError):
                linear(A, W.t(), workspace=ws[: need - 1], **args)
        graph = torch.cuda.CUDAGraph()
        X = A.clone()
        with torch.cuda.graph(graph):
            out = linear(X, W.t(), **args)
        X.copy_(ints(g, M, 400))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, (X.double() @ W.double().t()).float())


def test_refusals():
    z = lambda *s, t=I8: torch.zeros(*s, device="cuda").to(t)  # noqa: E731
    A, B, one = z(4, 16), z(8, 16).t(), torch.ones(16, device="cuda")
    ok = dict(scale_a=one[:4], scale_b=one[:8])
    for bad, err in [(lambda: linear(A, B), ValueError), (lambda: linear(A, B, scale_a=one[:4]), ValueError),
                     (lambda: linear(A, z(8, 16, t=E4M3).t(), **ok), TypeError), (lambda: linear(A, B, scale_a=one[:3], scale_b=one[:8]), ValueError),
                     (lambda: linear(A, B, scale_a=one[:4].half(), scale_b=one[:8]), TypeError),
                     (lambda: linear(A.to(torch.uint8), B.to(torch.uint8), **ok), TypeError),
                     (lambda: linear(A, B, out_dtype=I8, **ok), TypeError)]:
        with pytest.raises(err):
            bad()
    with pytest.raises(GemmError) as e:  # K has to be contiguous
        linear(A, z(16, 8), **ok)
    assert e.value.status == 2
