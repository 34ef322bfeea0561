"""GPU: sequences of dependent operator calls. Every kernel may start before the
one in front of it has ended, and kernels of one call that do not need each other
overlap; so sequences in which each call reads what the one before wrote, writes
what it read, or shares its workspace have to give, bit for bit, what the same
calls give with the device idle between them. Also: the whole step in a CUDA
graph, and matrices whose elements lie more than 2^31 elements apart."""
import pytest
import torch

from dense_gemm_gb300 import linear, linear_backward, rms_norm, rms_norm_backward, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, linear_ref

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def normal(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def same_in_a_row(step, state, rounds, repeats=3):
    """step(state, i, sync) for i in range(rounds), once with the device idle after
    every call and `repeats` times without: the state's tensors end the same."""
    start = [t.clone() for t in state]

    def run(sync):
        for t, s in zip(state, start):
            t.copy_(s)
        torch.cuda.synchronize()
        for i in range(rounds):
            step(state, i, sync)
        torch.cuda.synchronize()
        return [t.clone() for t in state]

    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(repeats):
        got = run(lambda: None)
        for k, (g, w) in enumerate(zip(got, want)):
            assert torch.equal(g, w), k


@pytest.mark.parametrize("kernel", ["pair", "split", "auto"])
@pytest.mark.parametrize("M,N", [(1, 512), (48, 1024), (300, 512), (1500, 768)])
def test_products_that_feed_each_other(kernel, M, N):
    W = normal(1, N, N, scale=N ** -0.5)

    def step(state, i, sync):
        a, b = state if i % 2 == 0 else state[::-1]
        linear(a, W, activation="gelu", residual=a, out=b, kernel=kernel)
        sync()

    x = normal(2, M, N)
    same_in_a_row(step, [x, torch.zeros_like(x)], 12)


@pytest.mark.parametrize("kernel", ["pair", "split"])
@pytest.mark.parametrize("b_t", [False, True])
def test_weights_written_by_the_call_before(kernel, b_t):
    """The second operand is what the norm has just written, so it must not be
    read, or kept from an earlier read, before the norm has ended."""
    M, K = 40, 512
    A, w = normal(3, M, K, scale=0.05), normal(4, K)

    def step(state, i, sync):
        src, y, c = state
        rms_norm(src, w, out=y)
        sync()
        linear(A, y.t() if b_t else y, out=c, kernel=kernel)
        sync()
        src[:M].copy_(c)
        sync()

    same_in_a_row(step, [normal(5, K, K), torch.zeros(K, K, device="cuda", dtype=BF16),
                         torch.zeros(M, K, device="cuda", dtype=BF16)], 10)


@pytest.mark.parametrize("tokens,width,hidden", [(1, 512, 1024), (64, 1024, 4096), (513, 520, 1000), (640, 257, 513),
                                                 (2048, 2048, 1024)])
def test_training_steps_sharing_buffers(tokens, width, hidden):
    """Forward and backward of norm, product and product again, in buffers that
    every step writes anew and one workspace for all of the gradients."""
    W1, W2 = normal(6, hidden, width, scale=width ** -0.5), normal(7, width, hidden, scale=hidden ** -0.5)
    w, bias = normal(8, width), normal(9, hidden, dtype=F32)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step(state, i, sync):
        x, r, u, pre, out, g1, g2, g3, dw, db = state
        n = rms_norm(x, w, residual=r, h_out=r, return_rstd=True)
        sync()
        linear(n.y, W1.t(), bias, activation="silu", out=u, pre=pre, workspace=ws)
        sync()
        linear(u, W2.t(), residual=r, out=out, workspace=ws)
        sync()
        du, dW2, _ = linear_backward(out, u, W2.t(), workspace=ws)
        sync()
        dy, dW1, dbias = linear_backward(du, n.y, W1.t(), pre=pre, activation="silu", need_bias=True, workspace=ws)
        sync()
        dx, dnorm = rms_norm_backward(dy, r, w, n.rstd, grad_h=out, out=dy)
        sync()
        for dst, src in ((g1, dW1.t()), (g2, dW2.t()), (g3, dx), (dw, dnorm), (db, dbias)):
            dst.copy_(src)
        x.copy_(dx / (1 + dx.abs()))
        r.copy_(out / (1 + out.abs()))
        sync()

    z = lambda *s, dtype=BF16: torch.zeros(*s, device="cuda", dtype=dtype)
    same_in_a_row(step, [normal(10, tokens, width), normal(11, tokens, width), z(tokens, hidden), z(tokens, hidden),
                         z(tokens, width), z(hidden, width), z(width, hidden), z(tokens, width), z(width, dtype=F32),
                         z(hidden, dtype=F32)], 4)


def test_step_in_a_graph():
    M, H, F = 200, 520, 1000
    W = normal(12, F, H, scale=0.05)
    w = normal(13, H)
    x = normal(14, M, H)
    g = normal(15, M, F)

    def step():
        n = rms_norm(x, w, return_rstd=True)
        c, pre = linear(n.y, W.t(), activation="gelu", return_pre=True)
        dy, dW, db = linear_backward(g, n.y, W.t(), pre=pre, activation="gelu", need_bias=True)
        dx, dw = rms_norm_backward(dy, x, w, n.rstd)
        return c, dW, db, dx, dw

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (16, 17, 18):
        x.copy_(normal(seed, M, H))
        g.copy_(normal(seed + 10, M, F))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ far apart

FAR = 800_000_000  # elements between rows: the fourth row starts past 2^31


def far(x, ld):
    """x in rows `ld` elements apart (the rest of the buffer is not initialised)."""
    buf = torch.empty((x.shape[0] - 1) * ld + x.shape[1], dtype=x.dtype, device="cuda")
    v = buf.as_strided(x.shape, (ld, 1))
    v.copy_(x)
    return v


@pytest.mark.parametrize("kernel", ["pair", "split"])
@pytest.mark.parametrize("ld", [FAR, FAR + 1])
def test_rows_past_32_bits(kernel, ld):
    M, N, K = 4, 136, 72
    A, B, R = normal(20, M, K), normal(21, K, N), normal(22, M, N)
    ref, pre_ref, ec, ep = linear_ref(A, B, None, "relu", R)
    out, pre = far(torch.zeros_like(R), ld), far(torch.zeros_like(R), ld)
    linear(far(A, ld), B, activation="relu", residual=far(R, ld), out=out, pre=pre, kernel=kernel)
    assert_close(out, ref, ec, "C")
    assert_close(pre, pre_ref, ep, "pre")
    # gradients: D's and A's rows, and B's where it is the wide one
    G = normal(23, M, N)
    dA, dB, db = linear_backward(far(G, ld), far(A, ld), B, pre=pre, activation="relu", need_bias=True, kernel=kernel)
    D = torch.where(pre.double() > 0, G.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    assert_close(dA, D @ B.double().t(), (N + 16) * 2.0 ** -23 * (D.abs() @ B.double().t().abs()), "dA")
    assert_close(dB, A.double().t() @ D, (M + 16) * 2.0 ** -23 * (A.double().t().abs() @ D.abs()), "dB")
    assert_close(db, D.sum(0), M * 2.0 ** -23 * D.abs().sum(0), "dbias")


@pytest.mark.parametrize("ld", [FAR, FAR + 1])
@pytest.mark.parametrize("width", [256, 1001])
def test_norm_rows_past_32_bits(ld, width):
    x, r, w = normal(24, 4, width), normal(25, 4, width), normal(26, width)
    y, h = far(torch.zeros_like(x), ld), far(torch.zeros_like(x), ld)
    n = rms_norm(far(x, ld), w, residual=far(r, ld), out=y, h_out=h, return_rstd=True)
    hd = x.double() + r.double()
    rstd = (hd.square().mean(1) + 1e-6).rsqrt()
    assert_close(h, hd, 2.0 ** -24 * hd.abs(), "h")
    assert_close(y, hd * rstd[:, None] * w.double(), 80 * 2.0 ** -24 * (hd * rstd[:, None] * w.double()).abs(), "y")
    want, dw = rms_norm_backward(x, h.contiguous(), w, n.rstd)
    got, dw2 = rms_norm_backward(far(x, ld), h, w, n.rstd, out=far(torch.zeros_like(x), ld))
    if ld % 8 == 0:  # the same kernel: the same bits
        assert torch.equal(got, want) and torch.equal(dw, dw2)
        return
    g, u = x.double() * w.double(), h.double() * n.rstd.double()[:, None]
    dx = n.rstd.double()[:, None] * (g - u * (g * u).mean(1, keepdim=True))
    size = n.rstd.double()[:, None] * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    assert_close(got, dx, 300 * 2.0 ** -24 * size, "dx")
    # four products of three factors each, summed in fp32
    assert_close(dw2, (x.double() * u).sum(0), 8 * 2.0 ** -24 * (x.double() * u).abs().sum(0), "dweight")


def test_more_than_32_bits_of_elements():
    """2.2e9 elements through the norm, the product and the norm's gradient; rows
    from all over are compared with the same rows on their own."""
    M, K, N = 270_000, 8192, 64
    x = torch.empty(M, K, device="cuda", dtype=BF16)
    g = torch.Generator(device="cuda").manual_seed(27)
    for i in range(0, M, 30_000):
        x[i:i + 30_000] = torch.randn(30_000, K, generator=g, device="cuda").to(BF16)
    w, B = normal(28, K), normal(29, K, N, scale=0.02)
    rows = torch.tensor([0, 1, 131_071, 262_143, 262_144, 262_145, M - 1], device="cuda")
    n = rms_norm(x, w, return_rstd=True)
    few = rms_norm(x[rows], w, return_rstd=True)
    hd = x[rows].double()
    y = hd * (hd.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    assert_close(n.y[rows], y, 80 * 2.0 ** -24 * y.abs(), "y")
    c = linear(n.y, B)
    ref, _, e, _ = linear_ref(n.y[rows], B)
    assert_close(c[rows], ref, e, "C")
    dx, dw = rms_norm_backward(n.y, x, w, n.rstd)
    gy, u = n.y[rows].double() * w.double(), hd * few.rstd.double()[:, None]
    want = few.rstd.double()[:, None] * (gy - u * (gy * u).mean(1, keepdim=True))
    size = few.rstd.double()[:, None] * (gy.abs() + u.abs() * (gy * u).abs().mean(1, keepdim=True))
    # rstd and the sums are 72 units of 2^-24 off at most, and each enters u and its mean
    assert_close(dx[rows], want, 300 * 2.0 ** -24 * size, "dx")
