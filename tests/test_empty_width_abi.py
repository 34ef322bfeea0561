"""CPU: rows of no values through the C ABI: the matrices may have no address, and the checks
that come before the GPU still hold."""
import ctypes as C

import pytest

from test_block_ops_abi import lib  # noqa: F401 - the fixture
from test_ops_abi import BF16, E4M3, F16, mat

I8 = 4


@pytest.fixture(scope="module")
def norms(lib):  # noqa: F811
    m, vp, i64 = C.POINTER(type(mat())), C.c_void_p, C.c_int64
    lib.gemm_rms_norm.argtypes = [m, m, vp, C.c_int32, m, m, vp, vp, i64, i64, C.c_float, vp]
    return lib


def test_nothing_to_write(norms):
    none = mat(None)
    for t in (F16, E4M3, I8):
        y = mat(None, t=t)
        assert norms.gemm_layer_norm(none, none, None, None, F16, y, none, None, None, None, 4, 0, 1e-5, None) == 0
        if t != I8:
            assert norms.gemm_rms_norm(none, none, None, F16, y, none, None, None, 4, 0, 1e-5, None) == 0
        if t != F16:
            assert norms.gemm_quantize_rows(none, y, None, 4, 0, None) == 0


def test_refusals(norms):
    none = mat(None)
    for s, mean, r in ((257, None, None), (None, 258, None), (None, None, 259)):
        assert norms.gemm_layer_norm(none, none, None, None, F16, mat(None, t=I8), none, s, mean, r, 4, 0, 1e-5, None) == 1
    assert norms.gemm_rms_norm(none, none, None, F16, none, none, None, 258, 4, 0, 1e-5, None) == 1
    assert norms.gemm_quantize_rows(none, mat(None, t=I8), 257, 4, 0, None) == 1
    assert norms.gemm_quantize_rows(none, mat(None, t=BF16), None, 4, 0, None) == 1
    assert norms.gemm_layer_norm(none, none, None, None, F16, none, none, None, None, None, 4, 0, -1.0, None) == 1
