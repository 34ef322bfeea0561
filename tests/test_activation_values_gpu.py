"""GPU: the activations and their slopes in fp32 at all 16-bit values up to 16,
against 64 bits, with bounds from the formulas in use (u = 2^-24, one rounding):

 * ex2.approx is off by 4 u of its value, rcp.approx by 2 u;
 * logistic(z) = 1 / (1 + 2^(-z log2 e)): 2 u of the exponent, so 2 |z| u, then
   4 + 1 + 2 u: relatively (2 |z| + 7) u;
 * what these two instructions give below 2^-126 they give as 0 (ftz), so the logistic
   is also off by up to 2^-126, absolutely;
 * the tanh form's z has 6 u of its own: (8 |z| + 7) u;
 * the normal distribution by Abramowitz & Stegun 26.2.17: absolutely 7.5e-8, and
   its evaluation: q = density * polynomial(t) with 1.5 x^2 + 8 u in the density, 54
   u in the polynomial's terms (4.5 times its value in magnitude at t = 1, 12
   roundings) and 65 in t (4 u, 16 times at t = 1). In the negative tail this is no
   relative bound: 7.5e-8 |x| is more than a tenth of gelu(x) below x = -4.9.
"""
import math

import pytest
import torch

from dense_gemm_gb300 import linear, linear_backward, sync_status
from gpu_util import require_gpu
from ops_util import act

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24
AS = 7.5e-8
FLUSH = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_gemm_gb300 import build
    build.build()
    yield
    assert sync_status() == 0


def values(dtype):
    """Every value of the type with 1e-30 <= |x| <= 16, and 0; an odd number of them."""
    x = torch.arange(-2 ** 15, 2 ** 15, device="cuda", dtype=torch.int32).to(torch.int16).view(dtype)
    f = x.float()
    keep = f.isfinite() & (f.abs() <= 16) & (f.abs() >= 1e-30)
    return torch.cat([x[keep], torch.zeros(1, device="cuda", dtype=dtype)])


def parts(x, name):
    """(logistic or Phi, its argument's magnitude, dz/dx) in float64."""
    if name == "gelu":
        return 0.5 * torch.special.erfc(-x * math.sqrt(0.5)), x.abs(), None
    if name == "silu":
        return torch.sigmoid(x), x.abs(), torch.ones_like(x)
    c = 2 * math.sqrt(2 / math.pi)
    z = c * (x + 0.044715 * x ** 3)
    return torch.sigmoid(z), z.abs(), c * (1 + 3 * 0.044715 * x ** 2)


def tail_error(x):
    q = 0.5 * torch.special.erfc(x.abs() * math.sqrt(0.5))
    return AS + q * (127 + 1.5 * x ** 2) * U


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kernel", ["pair", "split"])
@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_values(name, dtype, kernel):
    b = values(dtype)
    got = linear(torch.ones(1, 1, device="cuda", dtype=dtype), b[None, :], activation=name, out_dtype=F32, kernel=kernel)[0].double()
    x = b.double()
    want = act(x, name)
    if name == "relu":
        assert torch.equal(got, want)
        return
    s, z, _ = parts(x, name)
    if name == "gelu":
        bound = x.abs() * (tail_error(x) + 2 * U * s)
    else:
        bound = want.abs() * ((2 if name == "silu" else 8) * z + 8) * U + x.abs() * FLUSH
    bad = (got - want).abs() > 1.01 * bound + 1e-37
    assert not bad.any(), [(float(x[i]), float(got[i]), float(want[i])) for i in bad.nonzero()[:3, 0]]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes(name, dtype, odd):
    """dbias of one row of ones is D in fp32, before its rounding to 16 bits."""
    b = values(dtype)
    b = b if odd else b[b.numel() % 8:]
    one = torch.ones(1, b.numel(), device="cuda", dtype=dtype)
    got = linear_backward(one, one[:, :1], one, pre=b[None, :], activation=name, need_a=False, need_b=False, need_bias=True)[2].double()
    x = b.double()
    if name == "relu":
        assert torch.equal(got, (x > 0).double())
        return
    s, z, dz = parts(x, name)
    if name == "gelu":
        d = torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        want = s + x * d
        bound = tail_error(x) + (x * d).abs() * (1.5 * x * x + 8) * U + 2 * U * (s + (x * d).abs())
    else:
        want = s + x * s * (1 - s) * dz
        r = ((2 if name == "silu" else 8) * z + 7) * U
        bound = (s * r + (x * dz).abs() * (s * r * (1 - s) + s * (s * r + U)) + 6 * U * (x * s * (1 - s) * dz).abs()
                 + 2 * U * (s + (x * s * (1 - s) * dz).abs()) + (1 + (x * dz).abs()) * FLUSH)
    bad = (got - want).abs() > 1.01 * bound + 1e-37
    assert not bad.any(), [(float(x[i]), float(got[i]), float(want[i])) for i in bad.nonzero()[:3, 0]]
