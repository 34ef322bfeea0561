"""Plain 64-bit forms of the block operators and error bounds for their tests.

Bounds, derived from the arithmetic:
 * a sum of K products in fp32 on the tensor cores: every addition loses at most
   2^-23 of the sum of magnitudes, so |error| <= (K + 16) 2^-23 sum |a||b|;
 * an activation passes its argument's error on with a slope of at most 1.13
   (gelu's largest), and its own evaluation adds at most 2e-6 (1 + |x|): the fp32
   functions are within a few units in the last place (2^-24 = 6e-8 each),
   __expf's 2 + |1.2 x| of them at |x| < 20 included;
 * one rounding to the output's type: half a unit in its last place.
"""
import math

import torch

HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.float16, torch.bfloat16)}
TINY = {torch.float32: 1e-38, torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}


def act(x, name):
    if name == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if name == "gelu":
        return x * 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
    if name == "gelu_tanh":
        return x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    if name == "silu":
        return x * torch.sigmoid(x)
    return x


def rounding(ref, dtype):
    return HALF_ULP[dtype] * ref.abs() * 1.01 + TINY[dtype]


def sum_error(A, B):
    """Bound of a product's error in fp32, elementwise (A, B float64)."""
    K = A.shape[1]
    return (K + 16) * 2.0 ** -23 * (A.abs() @ B.abs())


def linear_ref(A, B, bias=None, activation="none", residual=None, scale_a=None, scale_b=None):
    """(C, pre, bound of C's error before rounding, bound of pre's) in float64."""
    A, B = A.double(), B.double()
    x = A @ B
    e = sum_error(A, B)
    if scale_a is not None:
        s = scale_a.double()[:, None] * scale_b.double()
        x, e = x * s, e * s.abs() + 3 * 2.0 ** -24 * (x * s).abs()
    if bias is not None:
        x = x + bias.double()
        e = e + 2.0 ** -24 * x.abs()
    c = act(x, activation)
    ec = e * 1.13 + (2e-6 * (1 + x.abs()) if activation not in ("none", "relu") else 0)
    if residual is not None:
        c = c + residual.double()
        ec = ec + 2.0 ** -24 * c.abs()
    return c, x, ec, e


def assert_close(got, ref, bound, what=""):
    """|got - ref| <= bound + one rounding to got's type, everywhere."""
    assert got.shape == ref.shape, what
    d = (got.double() - ref).abs()
    limit = bound + rounding(ref, got.dtype)
    bad = ~(d <= limit)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {d.numel()} values off, worst {float((d - limit).max()):.3e} over, at {bad.nonzero()[0].tolist()}"


def strided(x, ld=None, offset=0, transposed=False):
    """x [r, c] with rows (or, transposed, columns) `ld` elements apart, `offset`
    elements into a buffer of its own that is NaN (255 for 8-bit types) elsewhere."""
    y = x.t() if transposed else x
    r, c = y.shape
    ld = c if ld is None else ld
    n = offset + max(0, (r - 1) * ld + c) + 3
    if x.element_size() == 1:
        buf = torch.full((n,), 255, dtype=torch.uint8, device=x.device).view(x.dtype)
    else:
        buf = torch.full((n,), float("nan"), dtype=x.dtype, device=x.device)
    v = buf.as_strided((r, c), (ld, 1), offset)
    v.view(torch.uint8).copy_(y.contiguous().view(torch.uint8)) if x.element_size() == 1 else v.copy_(y)
    return v.t() if transposed else v


def outside_untouched(view):
    """Every element of the view's buffer that is not in the view is still NaN."""
    buf = torch.empty(0, dtype=view.dtype, device=view.device).set_(view.untyped_storage())
    mask = torch.ones(buf.numel(), dtype=torch.bool, device=view.device)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool(torch.isnan(buf[mask]).all())
