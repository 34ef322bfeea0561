"""GPU: the norm and its gradients on 16-bit rows that start off 16-byte boundaries
at the same place in every array (odd widths, offsets), where whole granules are
worked on and their foreign elements, NaN here, must neither count nor change."""
import pytest
import torch

from dense_gemm_gb300 import rms_norm, rms_norm_backward, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, outside_untouched, strided

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


def normal(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# one group and less, cut groups on both sides, one to four loads per thread, rows side
# by side, several rows per thread (more than 304 blocks' rows), one and two blocks per SM
SIZES = [(1, 1), (3, 5), (2, 8), (9, 9), (5, 255), (700, 33), (64, 1001), (2500, 257), (1300, 1002), (3, 2043), (305, 4095),
         (640, 2049), (620, 3999), (7, 6143), (310, 8185), (4, 8190), (160, 8193), (5, 16377), (330, 16370), (2, 32761)]
PLACES = [(0, 0), (3, 0), (0, 5), (8, 1), (1, 7)]  # gap between rows, offset of the first


def bound(width):  # of rstd, relative, as for the other layouts
    return (max(32, width / 1024) + 40) * 2.0 ** -24


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_forward(size, place, dtype):
    rows, width = size
    gap, offset = place
    put = lambda t: strided(t, width + gap, offset)
    x, r, w = normal(1, rows, width, dtype=dtype), normal(2, rows, width, dtype=dtype), normal(3, width, dtype=dtype)
    hd = x.double() + r.double()
    rstd = (hd.square().mean(1) + EPS).rsqrt()
    y, h = put(torch.zeros_like(x)), put(torch.zeros_like(x))
    n = rms_norm(put(x), w, residual=put(r), out=y, h_out=h, return_rstd=True)
    assert_close(h, hd, 2.0 ** -24 * hd.abs(), "h")
    ref = hd * rstd[:, None] * w.double()
    assert_close(y, ref, bound(width) * ref.abs(), "y")
    assert_close(n.rstd, rstd, bound(width) * rstd, "rstd")
    if (rows - 1) * gap + offset > 0:
        assert outside_untouched(y) and outside_untouched(h)
    # without a residual, and in 8 bits
    xd = x.double()
    rs = (xd.square().mean(1) + EPS).rsqrt()
    ref = xd * rs[:, None] * w.double()
    y = put(torch.zeros_like(x))
    rms_norm(put(x), w, out=y)
    assert_close(y, ref, bound(width) * ref.abs(), "y alone")
    q = strided(torch.zeros_like(x).to(E4M3), width + gap, offset)
    n = rms_norm(put(x), w, out=q, out_dtype=E4M3)
    top = ref.abs().amax(1)
    assert_close(n.scale, top / 448, 2 * bound(width) * top / 448, "scale")
    # half a unit of e4m3's three bits, or of its smallest step, in the scale's size
    d = (q.float().double() * n.scale.double()[:, None] - ref).abs()
    assert bool((d <= 1.001 * torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * (top / 448)[:, None])
                 + 3 * bound(width) * ref.abs()).all())


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("through", [False, True])
def test_backward(size, place, through):
    rows, width = size
    gap, offset = place
    dtype = BF16 if through else F16
    put = lambda t: strided(t, width + gap, offset)
    dy, h, w = normal(4, rows, width, dtype=dtype), normal(5, rows, width, dtype=dtype), normal(6, width, dtype=dtype)
    gh = normal(7, rows, width, dtype=dtype) if through else None
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx = put(torch.zeros_like(h))
    _, dw = rms_norm_backward(put(dy), put(h), w, rstd, grad_h=None if gh is None else put(gh), out=dx)
    rs = rstd.double()[:, None]
    u, g = h.double() * rs, dy.double() * w.double()
    mean = (g * u).mean(1, keepdim=True)
    ref = rs * (g - u * mean)
    size_ = rs * (g.abs() + u.abs() * (g * u).abs().mean(1, keepdim=True))
    if through:
        ref, size_ = ref + gh.double(), size_ + gh.double().abs()
    # a sum over the row: at most width / 256 / 8 + 16 additions deep, and a few roundings around it
    assert_close(dx, ref, (max(32, width / 1024) + 48) * 2.0 ** -24 * size_, "dx")
    terms = dy.double() * u
    # each block's rows one after the other, then the blocks' sums by 32 in turn
    assert_close(dw, terms.sum(0), (rows / 304 + 60) * 2.0 ** -24 * terms.abs().sum(0), "dweight")
    if (rows - 1) * gap + offset > 0:
        assert outside_untouched(dx)
    # dx in the gradient's own place
    own = put(dy)
    rms_norm_backward(own, put(h), w, rstd, grad_h=None if gh is None else put(gh), out=own)
    assert torch.equal(own, dx)


def test_gaps_of_nothing_but_nan_and_infinity():
    """A row of NaN or infinities next to the others changes none of them."""
    x, w = normal(8, 41, 1001, dtype=BF16), normal(9, 1001, dtype=BF16)
    want = rms_norm(x, w).y
    dwant, _ = rms_norm_backward(x, x, w, torch.ones(41, device="cuda"))
    bad = x.clone()
    bad[7], bad[23, 0], bad[30, -1] = float("nan"), float("inf"), float("-inf")
    got = rms_norm(bad, w).y
    dgot, _ = rms_norm_backward(bad, bad, w, torch.ones(41, device="cuda"))
    keep = [i for i in range(41) if i not in (7, 23, 30)]
    assert torch.equal(got[keep], want[keep]) and torch.equal(dgot[keep], dwant[keep])
    assert torch.isnan(got[7]).all()


@pytest.mark.parametrize("rows,width", [(700, 2056), (2500, 2304), (610, 8192), (615, 12296)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_many_rows(rows, width, dtype, with_residual):
    x, w = normal(10, rows, width, dtype=dtype), normal(11, width, dtype=dtype)
    r = normal(12, rows, width, dtype=dtype) if with_residual else None
    hd = x.double() + (r.double() if with_residual else 0)
    rstd = (hd.square().mean(1) + EPS).rsqrt()
    ref = hd * rstd[:, None] * w.double()
    n = rms_norm(x, w, residual=r, return_rstd=True)
    # h is the unrounded sum in fp32: half a unit of 2^-24 of it
    assert_close(n.y, ref, (bound(width) + 2.0 ** -24) * ref.abs(), "y")
    if with_residual:
        assert_close(n.h, hd, 2.0 ** -24 * hd.abs(), "h")
    n = rms_norm(x, w, residual=r, out_dtype=E4M3)
    top = ref.abs().amax(1)
    d = (n.y.float().double() * n.scale.double()[:, None] - ref).abs()
    assert bool((d <= 1.001 * torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * (top / 448)[:, None])
                 + 3 * (bound(width) + 2.0 ** -24) * ref.abs()).all())
