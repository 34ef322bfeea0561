"""GPU: gradients of layer norm whose rows hold NaNs or infinities. Rows are worked on side by side in
a block, and off 16-byte boundaries share granules: a row's values may reach its own dx and the column sums
only. And the sums beside fp32 weights, at the sizes of every form of the kernels."""
import pytest
import torch

from dense_gemm_gb300 import layer_norm, layer_norm_backward, sync_status
from gpu_util import require_gpu
from ops_util import assert_close

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24
SIZES = [(7, 64), (70, 257), (333, 1000), (700, 127), (20, 4096), (19, 4095), (333, 5001), (5, 16384), (3, 17000)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def normal(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_row_stays_in_its_row(size, dtype, bad):
    rows, width = size
    h, w, dy, dh = normal(1, rows, width, dtype=dtype), normal(2, width, dtype=dtype), normal(3, rows, width, dtype=dtype), normal(4, rows, width, dtype=dtype)
    clean = layer_norm(h, w, return_stats=True)
    want, _, want_db = layer_norm_backward(dy, h, w, clean.mean, clean.rstd, grad_h=dh)
    row = rows // 2
    others = torch.arange(rows, device="cuda") != row
    for place in (0, width // 2, width - 1):
        h2 = h.clone()
        h2[row, place] = bad
        n = layer_norm(h2, w, return_stats=True)
        assert torch.equal(n.y[others], clean.y[others]) and torch.equal(n.mean[others], clean.mean[others]) and n.y[row].isnan().all()
        dx, dw, db = layer_norm_backward(dy, h2, w, n.mean, n.rstd, grad_h=dh)
        assert torch.equal(dx[others], want[others]) and dx[row].isnan().all() and dw.isnan().all() and torch.equal(db, want_db)
        dy2 = dy.clone()
        dy2[row, place] = bad
        dx, dw, db = layer_norm_backward(dy2, h, w, clean.mean, clean.rstd, grad_h=dh)
        assert torch.equal(dx[others], want[others]) and not dx[row].isfinite().any()
        column = torch.arange(width, device="cuda") == place
        assert torch.equal(db[~column], want_db[~column]) and not db[place].isfinite() and not dw[place].isfinite() and dw[~column].isfinite().all()
        dh2 = dh.clone()
        dh2[row, place] = bad
        dx, _, db = layer_norm_backward(dy, h, w, clean.mean, clean.rstd, grad_h=dh2)
        differs = (dx != want) | dx.isnan()
        assert differs.sum() == 1 and not dx[row, place].isfinite() and torch.equal(db, want_db)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_sums_with_fp32_weights(size, dtype):
    rows, width = size
    h, w, dy = normal(1, rows, width, dtype=dtype), normal(2, width), normal(3, rows, width, dtype=dtype)
    n = layer_norm(h, w, return_stats=True)
    dx, dw, db = layer_norm_backward(dy, h, w, n.mean, n.rstd)
    r, c = n.rstd.double()[:, None], h.double() - n.mean.double()[:, None]
    g, u, T = dy.double() * w.double(), c * r, max(32, width / 1024) + 42
    m1, m2 = g.mean(1, keepdim=True), (g * u).mean(1, keepdim=True)
    e = r * U * (8 * (g.abs() + m1.abs() + (u * m2).abs()) + (T + 2) * (g.abs().mean(1, keepdim=True) + u.abs() * (g * u).abs().mean(1, keepdim=True)))
    assert_close(dx, r * (g - m1 - u * m2), e + 8 * U * dx.double().abs(), "dx")
    t = dy.double() * u
    assert_close(dw, t.sum(0), (rows + 8) * U * t.abs().sum(0), "dweight")
    assert_close(db, dy.double().sum(0), (rows + 2) * U * dy.double().abs().sum(0), "dbias")
    assert torch.equal(layer_norm_backward(dy, h, w, n.mean, n.rstd, need_weight=False)[2], db)
    assert torch.equal(layer_norm_backward(dy, h, w, n.mean, n.rstd, need_bias=False)[1], dw)
