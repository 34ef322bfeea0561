"""GPU: rows in 8 bits with a scale each against plain 64-bit forms. The factor t / a, its
product with a value and the scale are each within 2^-24 of the 64-bit ones, then the
value is rounded once."""
import pytest
import torch

from dense_gemm_gb300 import GemmError, quantize_rows, sync_status
from gpu_util import require_gpu
from ops_util import assert_close, strided

pytestmark = pytest.mark.gpu
F16, BF16, F32, E4M3, I8 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
TOP = {E4M3: 448, I8: 127}
U = 2.0 ** -24


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


def check(q, s, x):
    out = q.dtype
    top = x.double().abs().amax(1)
    scale = top / TOP[out]
    assert_close(s, scale, 2 * U * scale, "scale")
    v = x.double() / scale[:, None]
    near = (lambda z: z.float().to(E4M3).double()) if out == E4M3 else torch.round
    lo, hi = near(v * (1 - 3 * U)), near(v * (1 + 3 * U))
    g = q.double()
    assert ((g == lo) | (g == hi)).all()
    assert (g.abs().amax(1) == TOP[out]).all()


@pytest.mark.parametrize("size", [(1, 1), (1, 64), (3, 7), (5, 255), (7, 257), (33, 1000), (4, 4096), (9, 4095), (300, 640), (700, 5000), (700, 5001),
                                  (3, 16384), (2, 32768), (2, 33000), (1, 65537)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("out", [E4M3, I8])
def test_values(size, dtype, out):
    x = normal(size[0], *size, dtype=dtype, scale=3)
    q, s = quantize_rows(x, out)
    assert q.dtype == out and s.dtype == F32
    check(q, s, x)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("width", [64, 1001, 4096, 60000])
@pytest.mark.parametrize("out", [E4M3, I8])
def test_rows_that_hold_nothing_or_too_much(dtype, width, out):
    x = normal(3, 7, width, dtype=dtype)
    x[0] = 0
    x[1, width // 2] = float("nan")
    x[2, 5] = -float("inf")
    x[3] = 0
    x[3, width - 1] = torch.finfo(dtype).tiny
    x[4] = 0
    x[4, 1] = -torch.finfo(dtype).max
    q, s = quantize_rows(x, out)
    assert s[0] == 1 and (q[0].float() == 0).all()
    for k in (1, 2):
        assert s[k].isnan() and ((q[k] == 0).all() if out == I8 else q[k].float().isnan().all())
    if dtype == F16:  # 6e-5; the others' smallest numbers are below what a scale is made for
        assert q[3, -1].float() == TOP[out] and (q[3, :-1].float() == 0).all()
    else:
        assert s[3] == 1 and (q[3].float() == 0).all()
    assert q[4, 1].float() == -TOP[out] and q[4].float().abs().sum() == TOP[out] and s[4].isfinite()
    check(q[5:], s[5:], x[5:])


@pytest.mark.parametrize("pads", [(8, 0), (3, 1), (0, 5), (7, 3)])
@pytest.mark.parametrize("size", [(5, 256), (9, 1001), (3, 60001)])
@pytest.mark.parametrize("out", [E4M3, I8])
def test_strides_and_untouched_gaps(pads, size, out):
    rows, width = size
    pad, off = pads
    for dtype in (F16, F32):
        x = normal(1, rows, width, dtype=dtype)
        n = off + (rows - 1) * (width + pad) + width + 3
        buf = torch.full((n,), 99, dtype=torch.uint8, device="cuda")
        q = buf.view(out).as_strided((rows, width), (width + pad, 1), off)
        got, s = quantize_rows(strided(x, width + pad, off), out=q)
        assert got is q
        check(q, s, x)
        mask = torch.ones(n, dtype=torch.bool, device="cuda")
        mask.as_strided(q.shape, q.stride(), off).fill_(False)
        assert (buf[mask] == 99).all()


def test_ties_go_to_the_even_value():
    x = torch.tensor([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]], device="cuda")
    assert quantize_rows(x, I8)[0].tolist() == [[127, 0, 2, 2, 0, -2, -2, 126]]
    x = torch.tensor([[448, 17, 19, -17, 21, 0.001953125, 0.0009765625, 0.0029296875]], device="cuda")
    assert quantize_rows(x)[0].float().tolist() == [[448, 16, 20, -16, 20, 0.001953125, 0, 0.00390625]]


def test_empty_sizes_streams_and_refusals():
    x = normal(1, 4, 64, dtype=F16)
    q, s = quantize_rows(x[:0])
    assert q.shape == (0, 64) and s.shape == (0,)
    want = quantize_rows(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q, s = quantize_rows(x, stream=st)
    st.synchronize()
    assert torch.equal(q.float(), want[0].float()) and torch.equal(s, want[1])
    for bad in (lambda: quantize_rows(x.double()), lambda: quantize_rows(x, F16), lambda: quantize_rows(x[0]), lambda: quantize_rows(x, out=x)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: quantize_rows(x.cpu()), lambda: quantize_rows(x, out=torch.empty(4, 63, dtype=I8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: quantize_rows(x.t().contiguous().t()), lambda: quantize_rows(x[:1].expand(4, 64))):
        with pytest.raises(GemmError):
            bad()
