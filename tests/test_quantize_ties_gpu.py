"""GPU: 8-bit rows of 16-bit values at the edges of rounding. x t / a lies exactly halfway
between two 8-bit values for many x of a row (x = a / 2 in integers; with 448 = 7 * 64, rows
whose a is a multiple of 7 in 8-bit floats), and everywhere else it is further than 2^-20 of
its value from such an edge: numerators and denominators are whole numbers of at most 20 bits.
So the stored value is the one nearest to x t / a, ties to the even one, with no tolerance."""
import pytest
import torch

from dense_gemm_gb300 import quantize_rows, sync_status
from gpu_util import require_gpu
from ops_util import strided

pytestmark = pytest.mark.gpu
F16, BF16, E4M3, I8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int8
TOP = {E4M3: 448, I8: 127}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def every_quotient(dtype, exponent, step=1):
    """A row for each (step-th) significand of a, its largest value, with all values of the
    type in the 11 binades below it, both signs."""
    bits = 8 if dtype == BF16 else 11
    whole = torch.arange(1 << (bits - 1), 1 << bits, device="cuda", dtype=torch.float64)
    values = torch.cat([whole * 2.0 ** -k for k in range(11)])
    a = whole[::step, None]
    x = torch.where(values <= a, values, torch.zeros_like(values))
    return (torch.cat([a, x, -x], 1) * 2.0 ** exponent).to(dtype)


def nearest(x, out):
    x = x.double()
    v = x * TOP[out] / x.abs().amax(1, keepdim=True)  # the product is exact, so a tie's quotient is
    return v.float().to(E4M3).double() if out == E4M3 else torch.round(v)


@pytest.mark.parametrize("out", [E4M3, I8])
@pytest.mark.parametrize("dtype,exponent", [(BF16, 0), (BF16, 119), (BF16, -110), (F16, 4), (F16, 0)])
def test_every_value_is_the_nearest(dtype, exponent, out):
    step = 1 if dtype == BF16 else 7  # 7 and 1024 have no common factor but 1: all residues are met
    x = every_quotient(dtype, exponent, step)
    assert x.isfinite().all()
    want = nearest(x, out)
    rows, width = x.shape
    q, _ = quantize_rows(x, out)
    assert torch.equal(q.double(), want)
    few, _ = quantize_rows(x[:5], out)
    assert torch.equal(few.double(), want[:5])
    # rows at odd places, all the same, and values that lie at another place than their rows
    q, _ = quantize_rows(strided(x, width + 3, 1), out=torch.empty(rows, width + 3, dtype=out, device="cuda")[:, 1:width + 1])
    assert torch.equal(q.double(), want)
    q, _ = quantize_rows(strided(x, width + 5, 1), out=torch.empty(rows, width, dtype=out, device="cuda"))
    assert torch.equal(q.double(), want)


@pytest.mark.parametrize("out", [E4M3, I8])
@pytest.mark.parametrize("width", [40000, 70000])
def test_long_rows(width, out):
    g = torch.Generator(device="cuda").manual_seed(width)
    x = torch.randint(-255, 256, (9, width), generator=g, device="cuda").to(BF16)
    x[:, 7] = torch.tensor([254, 252, 250, 248, 224, 196, 255, 112, 98], device="cuda").to(BF16)
    x = x.clamp(-x[:, 7:8].abs(), x[:, 7:8].abs())
    assert torch.equal(quantize_rows(x, out)[0].double(), nearest(x, out))
