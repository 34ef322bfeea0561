"""GPU: the 8-bit norm on rows whose values are very small, zero or not finite,
through each of its kernels, against the definition in 64 bits."""
import pytest
import torch

from dense_gemm_gb300 import rms_norm, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn
TINY = 7.7e-34  # rows whose largest |y| is below are stored as zeros with scale 1


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


# width, offset of x's first element, of y's: values in registers (rows on 16-byte
# boundaries, and off them), through shared memory, and long rows
FORMS = [(64, 0, 0), (4096, 0, 0), (1001, 3, 3), (1001, 1, 0), (40000, 0, 0)]


def quantised(x, w, eps, offsets):
    ox, oy = offsets
    out = strided(torch.zeros(x.shape, device="cuda").to(E4M3), None, oy)
    n = rms_norm(strided(x, None, ox), w, eps=eps, out=out, out_dtype=E4M3)
    return out.float().double(), n.scale


def pattern(rows, width):
    """Rows of 1, 0, 1/2, 0, -1/4, 0 over and over: two of three rows end in a cut group."""
    p = torch.tensor([1, 0, 0.5, 0, -0.25, 0], device="cuda").repeat(width // 6 + 1)[:width]
    return p.expand(rows, width).clone()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("eps", [1e-6, 1e-12])
def test_small_rows_keep_their_values(form, dtype, eps):
    """mean(h^2) is far below eps, so y = w h / sqrt(eps) to 64 bits. A row's values
    are those of its quotients by its largest: 448, 0, 224 and -112 (exact in e4m3,
    and the quotients' error is a few 2^-24)."""
    width, *offsets = form
    tops = torch.tensor([8e-37, 1e-36, 1.3e-36, 1.4e-36, 1e-35, 1e-30], device="cuda").to(dtype)
    x = (pattern(6, width) * tops.float()[:, None]).to(dtype)
    q, scale = quantised(x, torch.ones(width, device="cuda", dtype=dtype), eps, offsets)
    a = tops.double() / eps ** 0.5
    assert bool((a > TINY).all())
    assert torch.equal(q, pattern(6, width).double() * 448)
    # rstd's and two products' roundings
    assert_close(scale, a / 448, 8 * 2.0 ** -24 * a / 448, "scale")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_small_weights_without_eps(form, dtype):
    """eps = 0: rows of magnitude 1e-4, 1e-3 and 1 under weights of 2^-110 (7.7e-34):
    w h down to 2e-38, y about 1.6e-33."""
    width, *offsets = form
    x = (pattern(3, width) * torch.tensor([1e-4, 1e-3, 1], device="cuda")[:, None]).to(dtype)
    w = torch.full((width,), 2.0 ** -110, device="cuda", dtype=dtype)
    q, scale = quantised(x, w, 0.0, offsets)
    h = x.double()
    a = (h / h.square().mean(1, keepdim=True).sqrt() * 2.0 ** -110).abs().amax(1)
    assert bool((a > TINY).all())
    assert torch.equal(q, pattern(3, width).double() * 448)
    # rstd of a sum of `width` squares: half of (terms per thread + tree) 2^-24
    assert_close(scale, a / 448, (max(32, width / 1024) + 48) * 2.0 ** -24 * a / 448, "scale")


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_zeros(form, dtype, eps):
    width, *offsets = form
    x = torch.ones(3, width, device="cuda", dtype=dtype)
    x[1] = 0
    q, scale = quantised(x, torch.ones(width, device="cuda", dtype=dtype), eps, offsets)
    assert scale[1] == 1 and bool((q[1] == 0).all()) and bool((q[[0, 2]] == 448).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_below_the_smallest_scale_are_zeros(form, dtype):
    width, *offsets = form
    x = (pattern(2, width) * 5e-37).to(dtype)  # a = 5e-34 at eps 1e-6
    q, scale = quantised(x, torch.ones(width, device="cuda", dtype=dtype), 1e-6, offsets)
    assert bool((scale == 1).all()) and bool((q == 0).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_an_infinite_weight_makes_rows_nan(form, dtype, bad):
    """y has an infinity (or a NaN, where h is zero) in that column."""
    width, *offsets = form
    x = torch.ones(3, width, device="cuda", dtype=dtype)
    x[1, width // 2] = 0
    w = torch.ones(width, device="cuda", dtype=dtype)
    w[width // 2] = bad
    q, scale = quantised(x, w, 1e-6, offsets)
    assert bool(scale.isnan().all()) and bool(q.isnan().all())
