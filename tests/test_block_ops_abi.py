"""The C ABI of layer norm, rows in 8 bits, gradients from them and integer products: every
declared symbol is exported, and arguments are checked on the host before a GPU is touched."""
import ctypes as C
import re

import pytest

from test_ops_abi import BF16, E4M3, F16, F32, HEADER, _Epilogue, _Matrix, epilogue, mat

I8 = 4
ONE = 256  # an address that is not read


@pytest.fixture(scope="module")
def lib():
    from dense_gemm_gb300 import build as b
    b.build()
    from dense_gemm_gb300 import binding
    lib = binding.load_library()
    m, e, vp = C.POINTER(_Matrix), C.POINTER(_Epilogue), C.c_void_p
    i64, i32, u32, u64, f32 = C.c_int64, C.c_int32, C.c_uint32, C.c_uint64, C.c_float
    pu64 = C.POINTER(u64)
    lib.gemm_linear.argtypes = [m, m, m, e, i64, i64, i64, u32, vp, u64, vp]
    lib.gemm_linear_workspace_size.argtypes = [m, m, i64, i64, i64, pu64]
    lib.gemm_layer_norm.argtypes = [m, m, vp, vp, i32, m, m, vp, vp, vp, i64, i64, f32, vp]
    lib.gemm_layer_norm_backward.argtypes = [m, m, vp, i32, vp, vp, m, m, vp, vp, i64, i64, vp, u64, vp]
    lib.gemm_layer_norm_backward_workspace_size.argtypes = [i64, i64, pu64]
    lib.gemm_quantize_rows.argtypes = [m, m, vp, i64, i64, vp]
    lib.gemm_saved_backward.argtypes = [m, m, vp, i32, m, m, vp, i32, m, m, vp, i64, i64, i64, u32, vp, u64, vp]
    lib.gemm_saved_backward_workspace_size.argtypes = [m, m, m, i32, i32, i64, i64, i64, pu64]
    return lib


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_(?:layer_norm|quantize|saved)\w*)\s*\(", text)))
    assert len(names) == 6, names
    for n in names:
        assert hasattr(lib, n), n


def _norm(lib, x=None, r=None, w=ONE, b=None, wt=F16, y=None, h=None, scale=None, mean=None, rstd=None, rows=4, width=8, eps=1e-5):
    return lib.gemm_layer_norm(x or mat(), r or mat(None), w, b, wt, y or mat(), h or mat(None), scale, mean, rstd, rows, width, eps, None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1), (dict(width=-1), 1), (dict(rows=2 ** 31), 1), (dict(x=mat(t=E4M3)), 1), (dict(x=mat(t=I8)), 1), (dict(y=mat(t=BF16)), 1),
    (dict(wt=BF16), 1), (dict(w=None), 1), (dict(w=257), 1), (dict(b=257), 1), (dict(b=258, wt=F32), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(scale=ONE), 1), (dict(y=mat(t=E4M3)), 1), (dict(y=mat(t=I8)), 1), (dict(y=mat(t=I8), scale=258), 1),
    (dict(mean=258), 1), (dict(rstd=257), 1), (dict(h=mat()), 1), (dict(r=mat(t=F32)), 1), (dict(r=mat(), h=mat(t=BF16)), 1), (dict(x=mat(data=None)), 1),
    (dict(x=mat(data=257)), 1), (dict(x=mat(r=7)), 1), (dict(y=mat(r=0)), 1), (dict(x=mat(r=16, c=2)), 2), (dict(y=mat(r=16, c=2)), 2)])
def test_layer_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want


def test_empty_norms(lib):
    assert _norm(lib, rows=0) == 0 and _norm(lib, width=0) == 0 and _norm(lib, rows=0, x=mat(data=None)) == 0


def _back(lib, g=None, h=None, w=ONE, wt=F16, mean=ONE, rstd=ONE, gh=None, dx=None, dw=None, db=None, rows=4, width=8, ws=None, nb=0):
    return lib.gemm_layer_norm_backward(g or mat(), h or mat(), w, wt, mean, rstd, gh or mat(None), dx or mat(), dw, db, rows, width, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(width=2 ** 31), dict(g=mat(t=E4M3)), dict(h=mat(t=BF16)), dict(dx=mat(t=F32)), dict(gh=mat(t=F32)), dict(wt=BF16), dict(w=None),
    dict(mean=None), dict(rstd=None), dict(mean=258), dict(rstd=257), dict(dw=258), dict(db=257), dict(dw=ONE), dict(db=ONE), dict(dw=ONE, ws=ONE, nb=255),
    dict(db=ONE, ws=264, nb=4096), dict(dx=mat(data=None)), dict(g=mat(r=7))])
def test_layer_norm_backward_refusals(lib, kw):
    assert _back(lib, **kw) == 1


def test_layer_norm_backward_workspace(lib):
    n = C.c_uint64()
    for rows, width, want in ((0, 8, 0), (4, 8, 4 * 8 * 8), (608, 100, 608 * 800), (10 ** 6, 100, 608 * 800)):
        assert lib.gemm_layer_norm_backward_workspace_size(rows, width, n) == 0 and n.value == want
    assert lib.gemm_layer_norm_backward_workspace_size(-1, 8, n) == 1


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), 1), (dict(x=mat(t=I8)), 1), (dict(q=mat(t=F16)), 1), (dict(scale=None), 1), (dict(scale=258), 1), (dict(x=mat(data=257)), 1),
    (dict(q=mat(t=I8, data=None)), 1), (dict(q=mat(t=I8, r=7)), 1), (dict(q=mat(t=E4M3, r=16, c=2)), 2), (dict(rows=0, scale=None), 0)])
def test_quantize_rows_refusals(lib, kw, want):
    a = dict(x=mat(), q=mat(t=I8), scale=ONE, rows=4, width=8) | kw
    assert lib.gemm_quantize_rows(a["x"], a["q"], a["scale"], a["rows"], a["width"], None) == want


def _saved(lib, G=None, A=None, sa=ONE, act_a=0, B=None, pre=None, sp=None, act=0, dA=None, dB=None, db=None, M=4, N=8, K=8, flags=0, ws=None, nb=0):
    return lib.gemm_saved_backward(G or mat(), A or mat(t=E4M3), sa, act_a, B or mat(), pre or mat(None), sp, act, dA or mat(None), dB or mat(None), db,
                                   M, N, K, flags, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), 1), (dict(sa=None), 1), (dict(A=mat()), 1), (dict(sa=258), 1), (dict(act_a=5), 1), (dict(act=9), 1), (dict(B=mat(t=BF16)), 1),
    (dict(G=mat(t=F32)), 1), (dict(G=mat(t=BF16)), 1), (dict(flags=3), 1), (dict(act=1, dA=mat()), 1), (dict(act=1, pre=mat(t=I8), dA=mat()), 1),
    (dict(act=1, pre=mat(), sp=ONE, dA=mat()), 1), (dict(act=1, pre=mat(t=BF16), dA=mat()), 1), (dict(act=1, pre=mat(t=E4M3, r=7), sp=ONE, dA=mat()), 1),
    (dict(dB=mat()), 1),  # no workspace for A'
    (dict(dB=mat(), ws=ONE, nb=511), 1), (dict(dB=mat(), ws=64, nb=512), 1), (dict(db=258), 1), (dict(dB=mat(t=E4M3), ws=ONE, nb=512), 1),
    (dict(A=mat(), sa=None, act_a=2), 2), (dict(A=mat(t=I8, r=1, c=8)), 2), (dict(A=mat(t=E4M3, r=16, c=2)), 2)])
def test_saved_backward_refusals(lib, kw, want):
    assert _saved(lib, **kw) == want


def test_saved_backward_workspace(lib):
    n = C.c_uint64()
    size = lambda *a: (lib.gemm_saved_backward_workspace_size(*a, n), n.value)  # noqa: E731
    a8 = mat(t=E4M3)
    assert size(mat(), a8, mat(), 0, 0, 4, 8, 8) == (0, 4 * 128)      # A' [4, 8], a row to a 128-byte line
    assert size(mat(), a8, mat(), 1, 0, 4, 8, 8) == (0, 2 * 4 * 128)  # and D
    assert size(mat(), mat(), mat(), 1, 0, 4, 8, 8) == (0, 4 * 128)   # A in 16 bits: D alone
    assert size(mat(), a8, mat(), 0, 0, 0, 8, 8) == (0, 0)
    assert size(mat(), a8, mat(t=BF16), 0, 0, 4, 8, 8)[0] == 1 and size(mat(), a8, mat(), 7, 0, 4, 8, 8)[0] == 1


def _linear(lib, A=None, B=None, Cm=None, ep=None, M=4, N=8, K=16, ws=None, nb=0):
    ep = ep or epilogue(scale_a=ONE, scale_b=ONE)
    return lib.gemm_linear(A or mat(t=I8, r=16), B or mat(t=I8, r=1, c=16), Cm or mat(), ep, M, N, K, 0, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(ep=epilogue()), 1), (dict(ep=epilogue(scale_a=ONE)), 1), (dict(ep=epilogue(scale_b=ONE)), 1), (dict(B=mat(t=E4M3, r=1, c=16)), 1),
    (dict(Cm=mat(t=I8)), 1), (dict(A=mat(t=I8, r=8), K=8, B=mat(t=I8, r=1, c=8)), 1),  # rows off 16-byte boundaries: no workspace
    (dict(B=mat(t=I8, r=16)), 2), (dict(A=mat(t=I8, r=1, c=16)), 2), (dict(M=0, ep=epilogue()), 0), (dict(N=0, ep=epilogue(scale_a=ONE)), 0)])
def test_integer_product_refusals(lib, kw, want):
    assert _linear(lib, **kw) == want


def test_integer_product_workspace(lib):
    n = C.c_uint64()
    size = lambda a, b, *s: (lib.gemm_linear_workspace_size(a, b, *s, n), n.value)  # noqa: E731
    a, b = mat(t=I8, r=4096), mat(t=I8, r=1, c=4096)
    assert size(a, b, 64, 4096, 4096) == (0, 0)                                # few rows: none
    assert size(a, b, 65, 4096, 4096) == (0, 65 * 4096 * 2)                    # A's copy in fp16
    assert size(a, b, 2048, 4096, 4096) == (0, (2048 + 4096) * 4096 * 2)       # both
    assert size(mat(t=I8, r=33), mat(t=I8, r=1, c=48), 3, 8, 33) == (0, 512)   # a copy on 128-byte lines
