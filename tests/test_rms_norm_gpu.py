"""GPU: the root-mean-square norm with the residual's addition, its 8-bit output
and its gradients against plain 64-bit forms.

Bounds: a row's sum of squares in fp32 is within (width / threads + 40) 2^-24 of
itself (all terms positive; a thread adds at most 32 terms, or width / 1024 in
the long form, before the tree), half of which reaches rstd; products and the
reciprocal root add a few 2^-24; then one rounding to the output's type.
"""
import pytest
import torch

from dense_gemm_gb300 import GemmError, linear, rms_norm, rms_norm_backward, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, linear_ref, outside_untouched, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


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


def ref(x, w, r=None):
    h = x.double() if r is None else x.double() + r.double()
    rstd = (h.square().mean(1) + EPS).rsqrt()
    return h * rstd[:, None] * w.double(), h, rstd


def rel(width):  # of rstd and so of y, before its rounding
    return (max(32, width / 1024) + 40) * 2.0 ** -24


SIZES = [(1, 1), (1, 64), (3, 7), (5, 255), (2, 256), (7, 257), (33, 1000), (4, 4096), (9, 4095), (2, 8192), (300, 640),
         (3, 16384), (2, 16383), (2, 32768), (2, 33000), (1, 65537)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_forward(size, dtype, with_residual):
    rows, width = size
    x = normal(rows, rows, width, dtype=dtype, scale=2)
    r = normal(width, rows, width, dtype=dtype) if with_residual else None
    for w in (normal(1, width, dtype=dtype), normal(1, width)):
        y, h, rstd = ref(x, w, r)
        got = rms_norm(x, w, residual=r, eps=EPS, return_rstd=True)
        assert got.scale is None and got.y.dtype == dtype
        assert_close(got.rstd, rstd, rstd * rel(width), "rstd")
        assert_close(got.y, y, y.abs() * rel(width), "y")
        if with_residual:
            assert_close(got.h, h, h.abs() * 2.0 ** -24, "h")
        else:
            assert got.h is None


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_eight_bits(size, dtype):
    """The stored value is within half a unit of e4m3 (1/16 of the value, 2^-10 where
    subnormal) of y / scale, the scale within rel of max|y| / 448."""
    rows, width = size
    x, r, w = normal(rows, rows, width, dtype=dtype), normal(2, rows, width, dtype=dtype, scale=3), normal(1, width, dtype=dtype)
    y, h, _ = ref(x, w, r)
    got = rms_norm(x, w, residual=r, eps=EPS, out_dtype=E4M3)
    scale = y.abs().amax(1) / 448
    assert_close(got.scale, scale, scale * (rel(width) + 2.0 ** -22), "scale")
    q, v = got.y.double(), y / scale[:, None]
    assert ((q - v).abs() <= v.abs() * (1 / 16 + 1e-5) + 2.0 ** -10 * 1.001).all()
    # all but values at a tie's edge round as the 64-bit quotient does
    assert ((q != v.float().to(E4M3).double()).double().mean()) <= 1e-4 + 2.0 / q.numel()
    assert (q.abs().amax(1) == 448).all()
    assert_close(got.h, h, h.abs() * 2.0 ** -24, "h")


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("width", [64, 4096, 1001, 40000])
def test_rows_that_hold_nothing_or_too_much(dtype, width):
    x = normal(3, 6, width, dtype=dtype)
    w = torch.ones(width, device="cuda")
    x[0] = 0
    x[1, width // 2] = float("nan")
    x[2, 5] = float("inf")
    x[3] = torch.finfo(dtype).tiny
    got = rms_norm(x, w, eps=EPS, out_dtype=E4M3)
    assert got.scale[0] == 1 and (got.y[0].float() == 0).all()
    assert got.scale[1].isnan() and got.y[1].float().isnan().all()
    assert got.scale[2].isnan() and got.y[2].float().isnan().all()
    assert not got.y[3:].float().isnan().any() and not got.scale[3:].isnan().any()
    y = rms_norm(x, w, eps=EPS).y
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 5].isnan() and (y[2, 6:] == 0).all()
    z = rms_norm(torch.zeros_like(x), w, eps=0.0)  # 0 * infinity
    assert z.y.isnan().all()


@pytest.mark.parametrize("pads", [(8, 0), (3, 1), (0, 5)])
@pytest.mark.parametrize("size", [(5, 256), (9, 1001), (3, 40001)])
@pytest.mark.parametrize("quant", [False, True])
def test_strides_and_untouched_gaps(pads, size, quant):
    rows, width = size
    pad, off = pads
    x, r, w = normal(1, rows, width, dtype=F16), normal(2, rows, width, dtype=F16), normal(3, width, dtype=F16)
    out = strided(torch.zeros(rows, width, dtype=F16, device="cuda"), width + pad, off)
    h = strided(torch.zeros(rows, width, dtype=F16, device="cuda"), width + 2 * pad, off)
    args = dict(residual=strided(r, width + pad, 2 * off), eps=EPS, h_out=h)
    plain = rms_norm(x, w, residual=r, eps=EPS, out_dtype=E4M3 if quant else None)
    if quant:
        got = rms_norm(strided(x, width + pad, off), w, out_dtype=E4M3, **args)
        # another order of the row's sum may move a value over a rounding edge
        assert (got.y.float() != plain.y.float()).float().mean() <= 1e-3
    else:
        rms_norm(strided(x, width + pad, off), w, out=out, **args)
        y = ref(x, w, r)[0]
        assert_close(out, y, y.abs() * rel(width), "y")
        assert outside_untouched(out)
    assert torch.equal(h, plain.h) and outside_untouched(h)


@pytest.mark.parametrize("width", [512, 1001, 33000])
def test_h_in_place(width):
    x, r, w = normal(1, 40, width, dtype=BF16), normal(2, 40, width, dtype=BF16), normal(3, width, dtype=BF16)
    want = rms_norm(x, w, residual=r)
    r2, x2 = r.clone(), x.clone()
    got = rms_norm(x, w, residual=r2, h_out=r2)
    assert got.h is r2 and torch.equal(r2, want.h) and torch.equal(got.y, want.y)
    got = rms_norm(x2, w, residual=r, h_out=x2)
    assert torch.equal(x2, want.h) and torch.equal(got.y, want.y)


# ------------------------------------------------------------------ gradients

BACK = [(1, 64), (3, 7), (2, 256), (70, 257), (333, 1000), (700, 128), (1500, 96), (20, 4096), (19, 4095), (4, 8192),
        (5, 16384), (3, 16383), (3, 17000), (700, 20000)]


@pytest.mark.parametrize("size", BACK)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("through", [False, True])
def test_backward(size, dtype, through):
    rows, width = size
    h, w = normal(1, rows, width, dtype=dtype, scale=2), normal(2, width, dtype=dtype)
    dy = normal(3, rows, width, dtype=dtype)
    dh = normal(4, rows, width, dtype=dtype) if through else None
    rstd = rms_norm(h, w, eps=EPS, return_rstd=True).rstd
    dx, dw = rms_norm_backward(dy, h, w, rstd, grad_h=dh)
    r = rstd.double()[:, None]
    u, g = h.double() * r, dy.double() * w.double()
    m = (g * u).mean(1, keepdim=True)
    want = r * (g - u * m) + (0 if dh is None else dh.double())
    # each term's products and the sum's order, then the additions
    e = 8 * 2.0 ** -24 * (r * (g.abs() + (u * m).abs()) + want.abs())
    e = e + r * u.abs() * rel(width) * (g * u).abs().mean(1, keepdim=True)
    assert_close(dx, want, e, "dx")
    terms = dy.double() * u
    assert_close(dw, terms.sum(0), (rows + 8) * 2.0 ** -24 * terms.abs().sum(0), "dweight")
    again, none = rms_norm_backward(dy, h, w, rstd, grad_h=dh, need_weight=False)
    assert none is None and torch.equal(again, dx)


def test_backward_against_differences():
    """Central differences of the fp32 forward pass in 64-bit sums: the step's square
    times the third derivative (about 1 for rows of unit scale) and the outputs'
    error 1e-6 sqrt(n) over the step."""
    rows, width, t = 6, 96, 2.0 ** -6
    h, w, R = normal(1, rows, width), normal(2, width), normal(3, rows, width)
    rstd = rms_norm(h, w, eps=EPS, return_rstd=True).rstd
    dx, dw = rms_norm_backward(R, h, w, rstd)

    def loss(h_, w_):
        return float((rms_norm(h_, w_, eps=EPS).y.double() * R.double()).sum())
    for which, grad in ((0, dx), (1, dw)):
        V = normal(7 + which, *grad.shape)
        hi = loss(h + t * V, w) if which == 0 else loss(h, w + t * V)
        lo = loss(h - t * V, w) if which == 0 else loss(h, w - t * V)
        got = float((grad.double() * V.double()).sum())
        assert abs((hi - lo) / (2 * t) - got) <= 5e-3 * float((grad.double() * V.double()).norm()) + 2e-3


@pytest.mark.parametrize("width", [512, 1001, 20000])
def test_backward_in_place_and_strides(width):
    h, w, dy, dh = (normal(1, 50, width, dtype=BF16), normal(2, width, dtype=BF16), normal(3, 50, width, dtype=BF16),
                    normal(4, 50, width, dtype=BF16))
    rstd = rms_norm(h, w, return_rstd=True).rstd
    dx, dw = rms_norm_backward(dy, h, w, rstd, grad_h=dh)
    a, b = dy.clone(), dh.clone()
    assert torch.equal(rms_norm_backward(a, h, w, rstd, grad_h=dh, out=a)[0], dx)
    assert torch.equal(rms_norm_backward(dy, h, w, rstd, grad_h=b, out=b)[0], dx)
    out = strided(torch.zeros_like(dx), width + 3, 1)
    got, dw2 = rms_norm_backward(strided(dy, width + 1, 1), strided(h, width + 5, 3), w, rstd, grad_h=strided(dh, width, 1), out=out)
    # the same formula with the row's sum in another order
    assert (got.float() - dx.float()).abs().max() <= 2.0 ** -7 * dx.float().abs().max() and outside_untouched(out)
    assert torch.allclose(dw, dw2, rtol=1e-4, atol=1e-4)


def test_norm_feeds_the_eight_bit_product():
    x, r, w = normal(1, 37, 512, dtype=BF16), normal(2, 37, 512, dtype=BF16), normal(3, 512, dtype=BF16)
    n = rms_norm(x, w, residual=r, out_dtype=E4M3)
    W = normal(4, 300, 512, scale=20).to(E4M3)
    sw = torch.rand(300, device="cuda") * 0.01 + 0.001
    got = linear(n.y, W.t(), scale_a=n.scale, scale_b=sw, activation="silu")
    c, _, ec, _ = linear_ref(n.y.float(), W.float().t(), None, "silu", None, n.scale, sw)
    assert_close(got, c, ec)


def test_empty_sizes_streams_and_refusals():
    x, w = normal(1, 4, 64, dtype=F16), normal(2, 64, dtype=F16)
    assert rms_norm(x[:0], w).y.shape == (0, 64)
    dx, dw = rms_norm_backward(x[:0], x[:0], w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = rms_norm(x, w, stream=s).y
    s.synchronize()
    assert torch.equal(y, rms_norm(x, w).y)
    for bad in (lambda: rms_norm(x.double(), w), lambda: rms_norm(x, w.to(BF16)), lambda: rms_norm(x, w, out_dtype=BF16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: rms_norm(x, w[:63]), lambda: rms_norm(x, w, residual=x[:3]), lambda: rms_norm(x, w, h_out=x),
                lambda: rms_norm(x.cpu(), w.cpu()), lambda: rms_norm_backward(x, x, w, torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: rms_norm(x, w, eps=-1.0), lambda: rms_norm(x, w, eps=float("nan")), lambda: rms_norm(x.t().contiguous().t(), w),
                lambda: rms_norm(x, w, residual=x[:1].expand(4, 64))):
        with pytest.raises(GemmError):
            bad()
