"""GPU: calls that depend on one another or run at the same time, and matrices past 2^31
elements. Launches may start before the ones in front of them have ended; a chain
whose calls read what the one before wrote, or overwrite what it read, has to give the
bits of the same calls with the device idle in between."""
import pytest
import torch

from dense_gemm_gb300 import layer_norm, layer_norm_backward, linear, linear_backward, quantize_rows, sync_status
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F16, BF16, F32, I8, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


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


def state(tokens, width, hidden):
    w1, s1 = quantize_rows(normal(1, hidden, width, scale=width ** -0.5), I8)
    w2, s2 = quantize_rows(normal(2, width, hidden, scale=hidden ** -0.5), I8)
    return dict(x=normal(3, tokens, width), r=normal(4, tokens, width), gain=normal(5, width), shift=normal(6, width), w1=w1, s1=s1, w2=w2, s2=s2,
                b1=normal(7, hidden, dtype=F32), q=torch.empty(tokens, hidden, dtype=I8, device="cuda"), ws=torch.empty(1 << 26, dtype=torch.uint8, device="cuda"),
                w16=normal(8, hidden, width, scale=width ** -0.5))


def steps(s, n, idle=False):
    """n times through the block, forward and back, in buffers that the calls share."""
    out = []

    def then():
        if idle:
            torch.cuda.synchronize()
    for _ in range(n):
        k = layer_norm(s["x"], s["gain"], s["shift"], residual=s["r"], out_dtype=I8, h_out=s["r"], return_stats=True)
        then()
        u = linear(k.y, s["w1"].t(), s["b1"], activation="gelu_tanh", scale_a=k.scale, scale_b=s["s1"], workspace=s["ws"])
        then()
        q, qs = quantize_rows(u, out=s["q"])
        then()
        linear(q, s["w2"].t(), scale_a=qs, scale_b=s["s2"], residual=s["r"], out=s["x"], workspace=s["ws"])
        then()
        da, dw, db = linear_backward(u, k.y, s["w16"].t(), scale_a=k.scale, pre=q, scale_pre=qs, activation="silu", need_bias=True, workspace=s["ws"])
        then()
        dx, dgain, dshift = layer_norm_backward(da, s["r"], s["gain"], k.mean, k.rstd, grad_h=s["x"], out=da, workspace=s["ws"])
        then()
        out += [s["x"].clone(), dw, db, dx, dgain, dshift]
    return out


@pytest.mark.parametrize("tokens,width,hidden", [(1, 512, 1024), (37, 264, 520), (300, 1001, 515), (70, 4096, 2048)])
def test_a_chain_gives_the_bits_of_its_calls_one_at_a_time(tokens, width, hidden):
    want = steps(state(tokens, width, hidden), 4, idle=True)
    for _ in range(5):
        got = steps(state(tokens, width, hidden), 4)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    sizes = [(1, 512, 1024), (70, 1024, 2048)]
    want = [steps(state(*z), 3, idle=True) for z in sizes]
    for _ in range(5):
        states = [state(*z) for z in sizes]
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream() for _ in sizes], []
        for s, st in zip(streams, states):
            with torch.cuda.stream(s):
                got.append(steps(st, 3))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs_on_two_streams():
    sizes = [(16, 512, 1024), (130, 264, 520)]
    want = [steps(state(*z), 2, idle=True) for z in sizes]
    graphs = []
    for z in sizes:
        st = state(*z)
        kept = {k: v.clone() for k, v in st.items()}
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = steps(st, 2)
        graphs.append((g, st, kept, out))
    streams = [torch.cuda.Stream() for _ in sizes]
    for _ in range(5):
        for _, st, kept, _ in graphs:
            for k in ("x", "r"):
                st[k].copy_(kept[k])
        torch.cuda.synchronize()
        for s, (g, _, _, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, _, _, out), w in zip(graphs, want):
            assert all(torch.equal(p, q) for p, q in zip(out, w))


def test_rows_past_two_to_the_31_elements():
    rows, width = 70001, 32768
    x = torch.empty(rows, width, dtype=BF16, device="cuda")
    x.view(-1)[: 1 << 20].normal_()
    x[-3:] = normal(1, 3, width)
    x[:1], mid = normal(2, 1, width), x[1:-3]
    mid.zero_()
    w, b = normal(3, width), normal(4, width)
    n = layer_norm(x, w, b, return_stats=True)
    last = layer_norm(x[-3:].clone(), w, b, return_stats=True)
    assert torch.equal(n.y[-3:], last.y) and torch.equal(n.mean[-3:], last.mean) and torch.equal(n.y[5], b)
    del n
    for out in (E4M3, I8):
        q, s = quantize_rows(x, out)
        ql, sl = quantize_rows(x[-3:].clone(), out)
        assert torch.equal(q[-3:].view(torch.uint8), ql.view(torch.uint8)) and torch.equal(s[-3:], sl) and s[7] == 1
        if out == E4M3:
            # all but the last rows count for nothing in dB
            B, G = normal(5, width, 64, scale=0.01), normal(6, rows, 64)
            scale = torch.zeros(rows, device="cuda")
            scale[-3:] = s[-3:]
            dB = linear_backward(G, q, B, scale_a=scale, need_a=False)[1]
            assert torch.equal(dB, linear_backward(G[-3:].clone(), ql, B, scale_a=sl, need_a=False)[1])
            del dB
        del q
    one = torch.ones(rows, device="cuda")
    W = torch.zeros(rows, width, dtype=I8, device="cuda")
    W[-2:] = torch.randint(-9, 10, (2, width), device="cuda")
    a = torch.randint(-9, 10, (1, width), device="cuda").to(I8)
    got = linear(a, W.t(), scale_a=one[:1], scale_b=one, out_dtype=F32)
    assert torch.equal(got[0, -2:].double(), (W[-2:].double() @ a[0].double())) and (got[0, :-2] == 0).all()
    del W
    n = layer_norm(x[-3:].clone(), w, b, return_stats=True)
    dx = layer_norm_backward(x, x, w, torch.zeros(rows, device="cuda"), one)[0]
    want = layer_norm_backward(x[-3:].clone(), x[-3:].clone(), w, torch.zeros(3, device="cuda"), one[:3])[0]
    assert torch.equal(dx[-3:], want)
