"""GPU: layer norm of rows of equal values, and of rows whose mean is far larger than their
deviation.

A row of equal values v has the mean v, no deviation and y = b, whatever the width: the mean
that is subtracted has to be v itself, since rstd = 1 / sqrt(eps) multiplies what is left
(with eps = 1e-12 a mean that is one unit of 1.0's last place off moves y by 0.06 w).

Elsewhere, u = 2^-24 and T as in test_layer_norm_gpu.py: the values less a first mean m1 are summed
again, so the mean is m1 plus T u mean|c| of error, rounded once, u |mean|. A centred value
carries that and three roundings of its own, y the row's rstd (half the variance's relative
error, 4 u for the root) and 4 u."""
import pytest
import torch

from dense_gemm_gb300 import layer_norm, layer_norm_backward, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
U = 2.0 ** -24
VALUES = [0.1, 1.0, -3.0, 100.0, 1234.5, -0.007, 31.7, 2.5e4, 6e-5]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


@pytest.mark.parametrize("width", [3, 768, 1000, 4095, 5000, 8192, 12000, 33000, 70000])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_a_row_of_equal_values_is_the_bias(width, dtype, with_residual):
    x = torch.tensor(VALUES, device="cuda").to(dtype)[:, None].expand(-1, width).contiguous()
    r = torch.tensor(VALUES[::-1], device="cuda").to(dtype)[:, None].expand(-1, width).contiguous() if with_residual else None
    h = x.float() if r is None else x.float() + r.float()
    g = torch.Generator(device="cuda").manual_seed(width)
    w, b = (torch.randn(width, generator=g, device="cuda").to(dtype) for _ in range(2))
    for eps in (1e-5, 1e-12):
        got = layer_norm(x, w, b, residual=r, eps=eps, return_stats=True)
        assert torch.equal(got.mean, h[:, 0])
        assert torch.equal(got.y, b.expand_as(x))
        assert_close(got.rstd, torch.full_like(got.rstd, eps).double().rsqrt(), 4 * U * got.rstd.double(), "rstd")
        for out in (E4M3, I8):
            got = layer_norm(x, w, None, residual=r, eps=eps, out_dtype=out)
            assert (got.scale == 1).all() and (got.y.float() == 0).all()
        apart = layer_norm(strided(x, width + 3, 1), w, b, residual=r, eps=eps)  # element by element
        assert torch.equal(apart.y, b.expand_as(x))
    assert layer_norm(x, w, b, residual=r, eps=0.0).y.isnan().all()  # 0 * infinity


@pytest.mark.parametrize("width", [768, 1000, 4095, 8192, 33000, 70000])
@pytest.mark.parametrize("offset,scale", [(100.0, 1.0), (1e4, 1.0), (-3e3, 0.01), (0.5, 1e-4)])
def test_the_mean_is_rounded_once(width, offset, scale):
    g = torch.Generator(device="cuda").manual_seed(width)
    x = offset + torch.randn(40, width, generator=g, device="cuda") * scale
    w, b = (torch.randn(width, generator=g, device="cuda") for _ in range(2))
    eps = 1e-12
    h, T = x.double(), max(32, width / 1024) + 42
    mean = h.mean(1, keepdim=True)
    c = h - mean
    size = c.abs().mean(1, keepdim=True)
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    e_m = U * mean.abs() + T * U * size
    e_c = e_m + 3 * U * (c.abs() + T * U * mean.abs())
    # the constant part of e_c adds its square only: the centred values' sum is about zero
    e_v = e_c.square().mean(1, keepdim=True) + 2 * T * U * (size * e_m + var) + 6 * U * var
    rel = e_v / (2 * (var + eps)) * 1.01 + 4 * U
    y = c * rstd * w.double() + b.double()
    e_y = w.double().abs() * rstd * (e_c + c.abs() * (rel + 4 * U)) + 2 * U * y.abs()
    for rows in (x, strided(x, width + 1, 0)):
        got = layer_norm(rows, w, b, eps=eps, return_stats=True)
        assert_close(got.mean, mean[:, 0], T * U * size[:, 0], "mean")
        assert_close(got.rstd, rstd[:, 0], (rstd * rel)[:, 0], "rstd")
        assert_close(got.y, y, e_y, "y")


@pytest.mark.parametrize("width", [768, 4095, 20000])
def test_gradients_of_equal_rows(width):
    """u = 0: dx = rstd (g - mean(g)), dweight = 0."""
    x = torch.tensor(VALUES, device="cuda")[:, None].expand(-1, width).contiguous()
    g = torch.Generator(device="cuda").manual_seed(1)
    w, dy = torch.randn(width, generator=g, device="cuda"), torch.randn(len(VALUES), width, generator=g, device="cuda")
    n = layer_norm(x, w, eps=1e-5, return_stats=True)
    dx, dw, db = layer_norm_backward(dy, x, w, n.mean, n.rstd)
    p = dy.double() * w.double()
    r, T = n.rstd.double()[:, None], max(32, width / 1024) + 42
    assert_close(dx, r * (p - p.mean(1, keepdim=True)), r * U * (8 * p.abs() + (T + 10) * p.abs().mean(1, keepdim=True)), "dx")
    assert (dw == 0).all()
    assert_close(db, dy.double().sum(0), 12 * U * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("rows,width", [(9, 64), (700, 520), (2000, 1024), (1000, 1001), (700, 2047), (2000, 4096), (40, 9000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", [None, I8])
def test_rows_with_and_without_a_correction_side_by_side(rows, width, dtype, out):
    """A block's rows do not wait for one another's correction, and none reaches another: a row has the same
    bits whatever stands beside it. (Rows change places with rows 8 k away: at an odd width a row starts
    width * row elements into a granule of 8, mod 8, and its threads' columns, and so the order of its
    sum, go by that.)"""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, width, generator=g, device="cuda")
    x[::2] += 50
    x[::5] = 7
    x = x.to(dtype)
    w, b = (torch.randn(width, generator=g, device="cuda").to(dtype) for _ in range(2))
    order = torch.arange(rows, device="cuda")
    for k in range(8):
        mine = order[k::8]
        order[k::8] = mine[torch.randperm(mine.numel(), generator=g, device="cuda")]
    one, other = (layer_norm(v.contiguous(), w, b, out_dtype=out, return_stats=True) for v in (x, x[order]))
    for p, q in zip(one, other):
        assert p is None or torch.equal(p[order], q)
