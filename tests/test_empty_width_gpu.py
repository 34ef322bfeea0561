"""GPU: rows of no values. Nothing of a row is stored, but what a row has beside its values is: the
scale 1 of rows of zeros, the mean 0 and 1 / sqrt(eps)."""
import pytest
import torch

from dense_gemm_gb300 import layer_norm, layer_norm_backward, linear, quantize_rows, rms_norm, rms_norm_backward, sync_status
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def leave_other_values(rows):
    """Blocks of the allocator that the calls' vectors will take hold something else."""
    held = [torch.full((rows,), float("nan"), device="cuda") for _ in range(16)]
    del held


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows", [1, 7, 1000, 70001])
def test_scales_and_statistics_are_defined(dtype, rows):
    x = torch.ones(rows, 8, dtype=dtype, device="cuda")[:, :0]
    w = torch.ones(0, dtype=dtype, device="cuda")
    for out in (E4M3, I8):
        leave_other_values(rows)
        q, s = quantize_rows(x, out)
        assert q.shape == (rows, 0) and (s == 1).all()
    rstd = torch.tensor(1e-3, device="cuda").double().rsqrt()
    for out in (None, E4M3, I8):
        for residual in (None, x):
            leave_other_values(rows)
            n = layer_norm(x, w, w, residual=residual, eps=1e-3, out_dtype=out, return_stats=True)
            assert (n.mean == 0).all() and ((n.rstd.double() - rstd).abs() < 1e-5).all()
            assert n.y.shape == (rows, 0) and (n.scale is None if out is None else (n.scale == 1).all())
    for out in (None, E4M3):
        leave_other_values(rows)
        n = rms_norm(x, w, eps=1e-3, out_dtype=out, return_rstd=True)
        assert ((n.rstd.double() - rstd).abs() < 1e-5).all() and (n.scale is None if out is None else (n.scale == 1).all())
    dx, dw, db = layer_norm_backward(x, x, w, torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda"))
    assert dx.shape == (rows, 0) and dw.shape == db.shape == (0,)
    dx, dw = rms_norm_backward(x, x, w, torch.ones(rows, device="cuda"))
    assert dx.shape == (rows, 0) and dw.shape == (0,)


def test_such_scales_go_into_a_product():
    """A sum of no products is 0: C is the bias."""
    leave_other_values(5)
    q, s = quantize_rows(torch.ones(5, 0, dtype=F16, device="cuda"), I8)
    leave_other_values(9)
    W, sw = quantize_rows(torch.ones(9, 0, dtype=F16, device="cuda"), I8)
    b = torch.randn(9, device="cuda")
    assert torch.equal(linear(q, W.t(), b, scale_a=s, scale_b=sw, out_dtype=F32), b.expand(5, 9))
