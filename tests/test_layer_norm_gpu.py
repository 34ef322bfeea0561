"""GPU: layer norm with the residual's addition, its 8-bit outputs and its gradients
against plain 64-bit forms.

Bounds, u = 2^-24. A sum of a row in fp32 is within T u of the sum of magnitudes, T =
max(32, width / 1024) + 42 (a thread adds at most 32 terms, or width / 1024 in the form
for long rows, then the tree). So the mean is off by e_m = (T + 1) u mean|h|, the addition of
the residual among it, a centred value c by e_m + u (|h| + |c|), the variance by
2 mean(|c| e_c) + T u var and rstd relatively by half of that over var + eps, plus 4 u
for the reciprocal root. y = w c rstd + b carries each of them once, and 4 u of its own.
Then one rounding to the output's type.
"""
import pytest
import torch

from dense_gemm_gb300 import GemmError, layer_norm, layer_norm_backward, linear, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, linear_ref, outside_untouched, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
EPS = 1e-5
U = 2.0 ** -24
TOP = {E4M3: 448, I8: 127}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def normal(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def terms(width):
    return max(32, width / 1024) + 42


def ref(x, w, b, r=None, eps=EPS):
    """((y, its bound), h, (mean, its bound), (rstd, its bound)) in 64 bits."""
    h = x.double() if r is None else x.double() + r.double()
    width, T = h.shape[1], terms(h.shape[1])
    mean = h.mean(1, keepdim=True)
    c = h - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    e_m = (T + 1) * U * h.abs().mean(1, keepdim=True)
    e_c = e_m + U * (h.abs() + c.abs())
    e_v = 2 * (c.abs() * e_c).mean(1, keepdim=True) + e_c.square().mean(1, keepdim=True) + T * U * var
    rel = e_v / (2 * (var + eps)) * 1.01 + 4 * U
    wd = w.double()
    y = c * rstd * wd + (0 if b is None else b.double())
    e_y = wd.abs() * rstd * (e_c + c.abs() * (rel + 4 * U)) + 2 * U * y.abs()
    return (y, e_y), h, (mean[:, 0], e_m[:, 0]), (rstd[:, 0], (rstd * rel)[:, 0])


SIZES = [(1, 1), (1, 64), (3, 7), (5, 255), (2, 256), (7, 257), (33, 1000), (4, 4096), (9, 4095), (2, 8192), (300, 640), (700, 5000),
         (3, 16384), (2, 16383), (2, 32768), (2, 33000), (1, 65537)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_forward(size, dtype, with_residual):
    rows, width = size
    x = normal(rows, rows, width, dtype=dtype, scale=2) + normal(9, rows, 1, dtype=dtype)
    r = normal(width, rows, width, dtype=dtype) if with_residual else None
    for w, b in ((normal(1, width, dtype=dtype), normal(2, width, dtype=dtype)), (normal(1, width), normal(2, width)),
                 (normal(1, width, dtype=dtype), None)):
        (y, e), h, (mean, e_m), (rstd, e_r) = ref(x, w, b, r)
        got = layer_norm(x, w, b, residual=r, eps=EPS, return_stats=True)
        assert got.scale is None and got.y.dtype == dtype
        assert_close(got.mean, mean, e_m, "mean")
        assert_close(got.rstd, rstd, e_r, "rstd")
        assert_close(got.y, y, e, "y")
        if with_residual:
            assert_close(got.h, h, h.abs() * U, "h")
        else:
            assert got.h is None


@pytest.mark.parametrize("width", [512, 1001, 9000])
@pytest.mark.parametrize("offset", [100.0, 10000.0])
def test_rows_whose_mean_is_far_larger_than_their_deviation(width, offset):
    """The mean square less the squared mean would leave rstd 2^-24 offset^2 off."""
    x, w, b = normal(1, 20, width) + offset, normal(2, width), normal(3, width)
    (y, e), _, (mean, e_m), (rstd, e_r) = ref(x, w, b)
    got = layer_norm(x, w, b, return_stats=True)
    assert_close(got.rstd, rstd, e_r, "rstd")
    assert_close(got.y, y, e, "y")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("out", [E4M3, I8])
def test_eight_bits(size, dtype, out):
    """A stored value is within half a step (e4m3 1/16 of the value, 2^-10 where subnormal;
    int8 one half) of y / scale, plus y's own error."""
    rows, width = size
    x, r = normal(rows, rows, width, dtype=dtype), normal(2, rows, width, dtype=dtype, scale=3)
    w, b = normal(1, width, dtype=dtype), normal(4, width, dtype=dtype)
    (y, e), h, _, _ = ref(x, w, b, r)
    got = layer_norm(x, w, b, residual=r, eps=EPS, out_dtype=out)
    top = y.abs().amax(1)
    scale = top / TOP[out]
    e_s = e.amax(1) / TOP[out]
    assert got.y.dtype == out
    assert_close(got.scale, scale, e_s + 3 * U * scale, "scale")
    q, v = got.y.double(), y / scale[:, None]
    e_v = (e + v.abs() * e_s[:, None] + 4 * U * y.abs()) / scale[:, None]
    step = v.abs() / 16 + 2.0 ** -10 if out == E4M3 else torch.full_like(v, 0.5)
    assert ((q - v).abs() <= step * 1.00001 + e_v * 1.1).all()
    # values far enough from a rounding's edge round as the 64-bit quotient does: all but a
    # share of 2 e_v over the values' spacing, far below 2 %, and of few values (21 in the
    # smallest matrix but one: 4.8 % each) one or two by chance
    lo, hi = v - e_v * 1.1, v + e_v * 1.1
    near = (lambda z: z.float().to(E4M3).double()) if out == E4M3 else torch.round
    sure = near(lo) == near(hi)
    assert (q[sure] == near(v)[sure]).all() and sure.double().mean() >= 0.98 - 2 / q.numel()
    assert (q.abs().amax(1) == TOP[out]).all()
    assert_close(got.h, h, h.abs() * U, "h")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("width", [64, 4096, 1001, 60000])
def test_rows_that_hold_nothing_or_too_much(dtype, width):
    x = normal(3, 6, width, dtype=dtype)
    w, b = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
    x[0] = 0
    x[1, width // 2] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 3
    for out in (E4M3, I8):
        got = layer_norm(x, w, b, eps=EPS, out_dtype=out)
        for k in (0, 3):  # equal values: y is b
            assert got.scale[k] == 1 and (got.y[k].float() == 0).all()
        for k in (1, 2):
            assert got.scale[k].isnan()
            assert (got.y[k] == 0).all() if out == I8 else got.y[k].float().isnan().all()
        assert not got.scale[4:].isnan().any() and (got.y[4:].float().abs().amax(1) == TOP[out]).all()
        some = layer_norm(x[:1], w, b + 2, eps=EPS, out_dtype=out)
        assert (some.y.float() == TOP[out]).all() and abs(float(some.scale) - 2 / TOP[out]) < 1e-7
    y = layer_norm(x, w, b, eps=EPS).y
    assert (y[0] == 0).all() and (y[3] == 0).all() and y[1:3].isnan().all() and not y[4:].isnan().any()
    assert layer_norm(x[3:4], w, b, eps=0.0).y.isnan().all()  # 0 * infinity


@pytest.mark.parametrize("pads", [(8, 0), (3, 1), (0, 5)])
@pytest.mark.parametrize("size", [(5, 256), (9, 1001), (3, 40001)])
@pytest.mark.parametrize("out", [None, E4M3, I8])
def test_strides_and_untouched_gaps(pads, size, out):
    rows, width = size
    pad, off = pads
    x, r, w, b = (normal(1, rows, width, dtype=F16), normal(2, rows, width, dtype=F16), normal(3, width, dtype=F16),
                  normal(4, width, dtype=F16))
    (y, e), ref_h, _, _ = ref(x, w, b, r)
    h = strided(torch.zeros(rows, width, dtype=F16, device="cuda"), width + 2 * pad, off)
    args = dict(residual=strided(r, width + pad, 2 * off), eps=EPS, h_out=h)
    if out is None:
        got = strided(torch.zeros(rows, width, dtype=F16, device="cuda"), width + pad, off)
        layer_norm(strided(x, width + pad, off), w, b, out=got, **args)
        assert_close(got, y, e, "y")
        assert outside_untouched(got)
    else:
        n = off + (rows - 1) * (width + pad) + width + 3
        buf = torch.full((n,), 99, dtype=torch.uint8, device="cuda")
        got = buf.view(out).as_strided((rows, width), (width + pad, 1), off)
        res = layer_norm(strided(x, width + pad, off), w, b, out=got, **args)
        assert res.y is got
        plain = layer_norm(x, w, b, residual=r, eps=EPS, out_dtype=out)
        # another order of the row's sum may move a value over a rounding edge
        assert (got.float() != plain.y.float()).float().mean() <= 1e-2
        mask = torch.ones(n, dtype=torch.bool, device="cuda")
        mask.as_strided(got.shape, got.stride(), off).fill_(False)
        assert (buf[mask] == 99).all()
    assert_close(h, ref_h, ref_h.abs() * U, "h")
    assert outside_untouched(h)


@pytest.mark.parametrize("width", [512, 1001, 33000, 60001])
def test_h_in_place(width):
    x, r, w, b = normal(1, 40, width, dtype=BF16), normal(2, 40, width, dtype=BF16), normal(3, width, dtype=BF16), normal(4, width, dtype=BF16)
    want = layer_norm(x, w, b, residual=r)
    r2, x2 = r.clone(), x.clone()
    got = layer_norm(x, w, b, residual=r2, h_out=r2)
    assert got.h is r2 and torch.equal(r2, want.h) and torch.equal(got.y, want.y)
    got = layer_norm(x2, w, b, residual=r, h_out=x2)
    assert torch.equal(x2, want.h) and torch.equal(got.y, want.y)


# ------------------------------------------------------------------ gradients
# The centred value of the given mean is one rounding off; the two row sums are within T u of
# their magnitudes' sums and reach dx through rstd / width; products and additions add 8 u of
# each term. A column's sum takes at most one addition per row.

BACK = [(1, 64), (3, 7), (2, 256), (70, 257), (333, 1000), (700, 128), (1500, 96), (20, 4096), (19, 4095), (700, 4095), (4, 8192), (333, 5001),
        (5, 16384), (3, 16383), (3, 17000), (700, 20000), (400, 12000)]


def back_ref(dy, h, w, mean, rstd, dh):
    width, T = h.shape[1], terms(h.shape[1])
    r, m = rstd.double()[:, None], mean.double()[:, None]
    c = h.double() - m
    u, g = c * r, dy.double() * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    want = r * (g - m1 - u * m2) + (0 if dh is None else dh.double())
    e = 8 * U * (r * (g.abs() + m1.abs() + (u * m2).abs()) + want.abs())
    e = e + r * (T + 2) * U * (g.abs().mean(1, keepdim=True) + u.abs() * (g * u).abs().mean(1, keepdim=True))
    return want, e, dy.double() * u


@pytest.mark.parametrize("size", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("through", [False, True])
def test_backward(size, dtype, through):
    rows, width = size
    h, w = normal(1, rows, width, dtype=dtype, scale=2) + normal(9, rows, 1, dtype=dtype), normal(2, width, dtype=dtype)
    dy = normal(3, rows, width, dtype=dtype)
    dh = normal(4, rows, width, dtype=dtype) if through else None
    n = layer_norm(h, w, eps=EPS, return_stats=True)
    dx, dw, db = layer_norm_backward(dy, h, w, n.mean, n.rstd, grad_h=dh)
    want, e, t = back_ref(dy, h, w, n.mean, n.rstd, dh)
    assert_close(dx, want, e, "dx")
    assert_close(dw, t.sum(0), (rows + 8) * U * t.abs().sum(0), "dweight")
    assert_close(db, dy.double().sum(0), (rows + 2) * U * dy.double().abs().sum(0), "dbias")
    again, none, db2 = layer_norm_backward(dy, h, w, n.mean, n.rstd, grad_h=dh, need_weight=False)
    assert none is None and torch.equal(again, dx) and torch.equal(db2, db)
    again, dw2, none = layer_norm_backward(dy, h, w, n.mean, n.rstd, grad_h=dh, need_bias=False)
    assert none is None and torch.equal(again, dx) and torch.equal(dw2, dw)
    again, none, none2 = layer_norm_backward(dy, h, w, n.mean, n.rstd, grad_h=dh, need_weight=False, need_bias=False)
    assert none is None and none2 is None and torch.equal(again, dx)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_backward_with_fp32_weights(dtype):
    for rows, width in ((50, 1024), (50, 1001), (20, 8192)):
        h, w, dy = normal(1, rows, width, dtype=dtype), normal(2, width), normal(3, rows, width, dtype=dtype)
        n = layer_norm(h, w, eps=EPS, return_stats=True)
        dx, dw, db = layer_norm_backward(dy, h, w, n.mean, n.rstd)
        want, e, t = back_ref(dy, h, w, n.mean, n.rstd, None)
        assert_close(dx, want, e, "dx")
        assert_close(dw, t.sum(0), (rows + 8) * U * t.abs().sum(0), "dweight")


def test_backward_against_differences():
    """Central differences of the fp32 forward pass in 64-bit sums: the step's square
    times the third derivative (about 1 for rows of unit scale) and the outputs'
    error 1e-6 sqrt(n) over the step."""
    rows, width, t = 6, 96, 2.0 ** -6
    h, w, b, R = normal(1, rows, width), normal(2, width), normal(5, width), normal(3, rows, width)
    n = layer_norm(h, w, b, eps=EPS, return_stats=True)
    grads = layer_norm_backward(R, h, w, n.mean, n.rstd)

    def loss(h_, w_, b_):
        return float((layer_norm(h_, w_, b_, eps=EPS).y.double() * R.double()).sum())
    for which, grad in enumerate(grads):
        V = normal(7 + which, *grad.shape)
        hi, lo = [h, w, b], [h, w, b]
        hi[which], lo[which] = hi[which] + t * V, lo[which] - t * V
        got = float((grad.double() * V.double()).sum())
        assert abs((loss(*hi) - loss(*lo)) / (2 * t) - got) <= 5e-3 * float((grad.double() * V.double()).norm()) + 2e-3


@pytest.mark.parametrize("width", [512, 1001, 20000])
def test_backward_in_place_and_strides(width):
    h, w, dy, dh = (normal(1, 50, width, dtype=BF16), normal(2, width, dtype=BF16), normal(3, 50, width, dtype=BF16),
                    normal(4, 50, width, dtype=BF16))
    n = layer_norm(h, w, return_stats=True)
    dx, dw, db = layer_norm_backward(dy, h, w, n.mean, n.rstd, grad_h=dh)
    a, b = dy.clone(), dh.clone()
    for got in (layer_norm_backward(a, h, w, n.mean, n.rstd, grad_h=dh, out=a), layer_norm_backward(dy, h, w, n.mean, n.rstd, grad_h=b, out=b)):
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    out = strided(torch.zeros_like(dx), width + 3, 1)
    got, dw2, db2 = layer_norm_backward(strided(dy, width + 1, 1), strided(h, width + 5, 3), w, n.mean, n.rstd,
                                        grad_h=strided(dh, width, 1), out=out)
    want, e, t = back_ref(dy, h, w, n.mean, n.rstd, dh)
    assert_close(got, want, e, "dx")
    assert outside_untouched(out)
    assert_close(dw2, t.sum(0), 58 * U * t.abs().sum(0), "dweight")
    assert_close(db2, dy.double().sum(0), 52 * U * dy.double().abs().sum(0), "dbias")


def test_norm_feeds_the_eight_bit_products():
    x, r, w, b = normal(1, 37, 512, dtype=BF16), normal(2, 37, 512, dtype=BF16), normal(3, 512, dtype=BF16), normal(6, 512, dtype=BF16)
    sw = torch.rand(300, device="cuda") * 0.01 + 0.001
    for out in (E4M3, I8):
        n = layer_norm(x, w, b, residual=r, out_dtype=out)
        W = normal(4, 300, 512, scale=20).to(out)
        got = linear(n.y, W.t(), scale_a=n.scale, scale_b=sw, activation="silu")
        c, _, ec, _ = linear_ref(n.y.float(), W.float().t(), None, "silu", None, n.scale, sw)
        assert_close(got, c, ec)


def test_empty_sizes_streams_graphs_and_refusals():
    x, w, b = normal(1, 4, 64, dtype=F16), normal(2, 64, dtype=F16), normal(3, 64, dtype=F16)
    none = torch.empty(0, device="cuda")
    assert layer_norm(x[:0], w, b).y.shape == (0, 64)
    dx, dw, db = layer_norm_backward(x[:0], x[:0], w, none, none)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    want = layer_norm(x, w, b, return_stats=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = layer_norm(x, w, b, stream=s).y
    s.synchronize()
    assert torch.equal(y, want.y)
    grads = layer_norm_backward(x, x, w, want.mean, want.rstd)
    graph = torch.cuda.CUDAGraph()
    static = x.clone()
    with torch.cuda.graph(graph):
        n = layer_norm(static, w, b, return_stats=True)
        captured = layer_norm_backward(static, static, w, n.mean, n.rstd)
    static.copy_(x.flip(0))
    graph.replay()
    static.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n.y, want.y) and all(torch.equal(p, q) for p, q in zip(captured, grads))
    one = torch.ones(4, device="cuda")
    for bad in (lambda: layer_norm(x.double(), w, b), lambda: layer_norm(x, w.to(BF16)), lambda: layer_norm(x, w, b.float()),
                lambda: layer_norm(x, w, b, out_dtype=BF16), lambda: layer_norm(x, w.float(), b)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: layer_norm(x, w[:63]), lambda: layer_norm(x, w, b[:63]), lambda: layer_norm(x, w, residual=x[:3]),
                lambda: layer_norm(x, w, h_out=x), lambda: layer_norm(x.cpu(), w.cpu()),
                lambda: layer_norm_backward(x, x, w, one[:3], one), lambda: layer_norm_backward(x, x, w, one, one[:3]),
                lambda: layer_norm_backward(x, x, w, one, one, workspace=torch.empty(1, device="cuda").expand(4096))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: layer_norm(x, w, eps=-1.0), lambda: layer_norm(x, w, eps=float("nan")), lambda: layer_norm(x.t().contiguous().t(), w),
                lambda: layer_norm(x, w, residual=x[:1].expand(4, 64)), lambda: layer_norm_backward(x, x, w, one, one, workspace=one)):
        with pytest.raises(GemmError):
            bad()
