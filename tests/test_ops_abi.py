"""The operators' C ABI: every declared symbol is exported, and arguments are
checked on the host before a GPU is touched."""
import ctypes as C
import os
import re

import pytest

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "gemm_ops.h")
F32, F16, BF16, E4M3 = 0, 1, 2, 3


class _Matrix(C.Structure):  # gemm_matrix_t
    _fields_ = [("data", C.c_void_p), ("stride_row", C.c_int64), ("stride_col", C.c_int64), ("type", C.c_int32)]


class _Epilogue(C.Structure):  # gemm_epilogue_t
    _fields_ = [("bias", C.c_void_p), ("bias_type", C.c_int32), ("activation", C.c_int32), ("scale_a", C.c_void_p),
                ("scale_b", C.c_void_p), ("residual", _Matrix), ("pre", _Matrix)]


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
    lib.gemm_linear_backward.argtypes = [m, m, m, m, i32, m, m, vp, i64, i64, i64, u32, vp, u64, vp]
    lib.gemm_linear_backward_workspace_size.argtypes = [m, m, m, i32, i32, i64, i64, i64, pu64]
    lib.gemm_rms_norm.argtypes = [m, m, vp, i32, m, m, vp, vp, i64, i64, f32, vp]
    lib.gemm_rms_norm_backward.argtypes = [m, m, vp, i32, vp, m, m, vp, i64, i64, vp, u64, vp]
    lib.gemm_rms_norm_backward_workspace_size.argtypes = [i64, i64, pu64]
    return lib


def mat(data=256, r=8, c=1, t=F16):
    return _Matrix(data, r, c, t)


def epilogue(**kw):
    e = _Epilogue(None, 0, 0, None, None, mat(None), mat(None))
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def test_library_exports_every_declared_symbol(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_(?:linear|rms_norm)\w*)\s*\(", text)))
    assert len(names) == 7, names
    for n in names:
        assert hasattr(lib, n), n


def _linear(lib, A=None, B=None, Cm=None, ep=None, M=4, N=8, K=8, flags=0, ws=None, nbytes=0):
    return lib.gemm_linear(A or mat(), B or mat(), Cm or mat(), ep or epilogue(), M, N, K, flags, ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=2 ** 31), dict(flags=3), dict(flags=4),
    dict(A=mat(t=E4M3)), dict(A=mat(t=F32), B=mat(t=F32)), dict(A=mat(t=9), B=mat(t=9)), dict(Cm=mat(t=E4M3)), dict(Cm=mat(t=-1)),
    dict(A=mat(r=0)), dict(B=mat(c=-1)), dict(A=mat(data=257)), dict(Cm=mat(data=258, t=F32)), dict(Cm=mat(data=None)),
    dict(A=mat(data=None)), dict(Cm=mat(r=7)),
    dict(ep=epilogue(activation=5)), dict(ep=epilogue(activation=-1)), dict(ep=epilogue(bias=256, bias_type=BF16)),
    dict(ep=epilogue(bias=257, bias_type=F16)), dict(ep=epilogue(scale_a=256)), dict(ep=epilogue(scale_a=256, scale_b=256)),
    dict(A=mat(t=E4M3), B=mat(t=E4M3, r=1, c=16)), dict(ep=epilogue(residual=mat(t=F32))), dict(ep=epilogue(residual=mat(r=4))),
    dict(ep=epilogue(pre=mat(data=129)))])
def test_linear_refuses_bad_arguments(lib, kw):
    assert _linear(lib, **kw) == 1


@pytest.mark.parametrize("kw", [dict(A=mat(r=16, c=2)), dict(B=mat(r=16, c=2)), dict(Cm=mat(r=16, c=2)),
                                dict(A=mat(t=E4M3, r=16), B=mat(t=E4M3, r=16), ep=epilogue(scale_a=256, scale_b=256))])
def test_linear_refuses_layouts_it_does_not_take(lib, kw):
    assert _linear(lib, **kw) == 2


def test_linear_empty_problems_and_workspace(lib):
    assert _linear(lib, M=0) == 0 and _linear(lib, N=0) == 0
    n = C.c_uint64(7)
    assert lib.gemm_linear_workspace_size(mat(), mat(), 4, 8, 8, n) == 0 and n.value == 0
    # A [4, 9] with rows of 9 elements: copied onto 128-byte lines; B [9, 8] stays
    a = mat(r=9)
    assert lib.gemm_linear_workspace_size(a, mat(), 4, 8, 9, n) == 0 and n.value == 4 * 128
    # both: each copy from a 256-byte boundary
    assert lib.gemm_linear_workspace_size(a, mat(r=1, c=9), 3, 8, 9, n) == 0 and n.value == 512 + 8 * 128
    # a single row needs no stride, only an aligned base
    assert lib.gemm_linear_workspace_size(mat(r=9), mat(), 1, 8, 9, n) == 0 and n.value == 0
    assert lib.gemm_linear_workspace_size(mat(data=258, r=9), mat(), 1, 8, 9, n) == 0 and n.value == 256
    assert _linear(lib, A=a, K=9) == 1                                   # no workspace
    assert _linear(lib, A=a, K=9, ws=256, nbytes=511) == 1               # too small
    assert _linear(lib, A=a, K=9, ws=64, nbytes=512) == 1                # misaligned
    assert lib.gemm_linear_workspace_size(mat(), mat(), -1, 8, 8, n) == 1


def _backward(lib, G=None, A=None, B=None, pre=None, act=0, dA=None, dB=None, db=None, M=4, N=8, K=8, flags=0, ws=None, nb=0):
    return lib.gemm_linear_backward(G or mat(), A or mat(), B or mat(), pre or mat(None), act, dA or mat(None), dB or mat(None),
                                    db, M, N, K, flags, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), 1), (dict(G=mat(t=BF16)), 1), (dict(G=mat(data=None), dA=mat()), 1), (dict(act=1, dA=mat()), 1),
    (dict(act=9), 1), (dict(dA=mat(t=E4M3)), 1), (dict(dA=mat(r=7)), 1), (dict(db=258), 1), (dict(flags=3), 1),
    (dict(act=1, pre=mat(t=BF16), dA=mat()), 1), (dict(act=1, pre=mat(), dA=mat()), 1),  # no workspace for D
    (dict(A=mat(t=E4M3), B=mat(t=E4M3, r=1, c=8), G=mat(t=E4M3)), 2), (dict(G=mat(r=16, c=2), dA=mat()), 2),
    (dict(dA=mat(r=16, c=2)), 2), (dict(B=mat(r=16, c=2), dA=mat()), 2)])
def test_linear_backward_refusals(lib, kw, want):
    assert _backward(lib, **kw) == want


def test_linear_backward_workspace(lib):
    n = C.c_uint64()
    size = lambda *a: (lib.gemm_linear_backward_workspace_size(*a, n), n.value)  # noqa: E731
    assert size(mat(), mat(), mat(), 0, 0, 4, 8, 8) == (0, 0)
    assert size(mat(), mat(), mat(), 2, 0, 4, 8, 8) == (0, 4 * 128)                    # D
    assert size(mat(r=8), mat(), mat(), 2, 1, 130, 8, 8) == (0, 130 * 128 + 768)       # and 17 blocks of 8 rows' sums of 8 columns
    assert size(mat(r=9), mat(), mat(r=9), 0, 0, 4, 9, 8)[1] == 4 * 128 + 1024         # G and B copied


def test_rms_norm_refusals(lib):
    def norm(x=None, r=None, w=256, wt=F16, y=None, h=None, scale=None, rstd=None, rows=4, width=8, eps=1e-6):
        return lib.gemm_rms_norm(x or mat(), r or mat(None), w, wt, y or mat(), h or mat(None), scale, rstd, rows, width, eps, None)
    for kw in (dict(rows=-1), dict(width=2 ** 31), dict(x=mat(t=E4M3)), dict(y=mat(t=BF16)), dict(wt=BF16), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(y=mat(t=E4M3)), dict(scale=256), dict(w=None), dict(h=mat()),
               dict(x=mat(r=7)), dict(x=mat(data=257)), dict(rstd=258), dict(w=257), dict(r=mat(t=F32)), dict(r=mat(r=0))):
        assert norm(**kw) == 1, kw
    assert norm(x=mat(r=16, c=2)) == 2
    assert norm(rows=0) == 0 and norm(width=0) == 0

    def back(g=None, h=None, w=256, wt=F16, rstd=256, gh=None, dx=None, dw=None, rows=4, width=8, ws=None, nb=0):
        return lib.gemm_rms_norm_backward(g or mat(), h or mat(), w, wt, rstd, gh or mat(None), dx or mat(), dw, rows, width, ws, nb,
                                          None)
    for kw in (dict(rows=-1), dict(g=mat(t=E4M3)), dict(h=mat(t=BF16)), dict(wt=BF16), dict(rstd=None), dict(dw=256), dict(dw=258),
               dict(dw=256, ws=256, nb=127), dict(dw=256, ws=264, nb=128), dict(dx=mat(data=None)), dict(gh=mat(r=4))):
        assert back(**kw) == 1, kw
    assert back(dx=mat(r=16, c=2)) == 2
    n = C.c_uint64()
    assert lib.gemm_rms_norm_backward_workspace_size(4, 8, n) == 0 and n.value == 128
    assert lib.gemm_rms_norm_backward_workspace_size(1 << 20, 8, n) == 0 and n.value == 608 * 32
    assert lib.gemm_rms_norm_backward_workspace_size(-1, 8, n) == 1


def test_binding_checks_before_the_library():
    """The Python entry points name what is wrong with host tensors, types, shapes
    and keywords without a GPU."""
    import torch
    from dense_gemm_gb300 import linear, linear_backward, rms_norm, rms_norm_backward
    z = lambda *s, t=torch.float16: torch.zeros(*s).to(t)  # noqa: E731
    A, B, E = z(4, 8), z(8, 16), torch.float8_e4m3fn
    with pytest.raises(ValueError, match="CUDA"):
        linear(A, B)
    with pytest.raises(ValueError, match="chain"):
        linear(A, z(9, 16))
    with pytest.raises(ValueError, match="activation"):
        linear(A, B, activation="tanh")
    with pytest.raises(ValueError, match="scale"):
        linear(A.to(E), B.to(E))
    for bad in (lambda: linear(A, z(8, 16, t=torch.bfloat16)), lambda: linear(A.float(), B.float()), lambda: linear(A, 3),
                lambda: linear(None, B), lambda: linear(A, B, out_dtype=torch.int32), lambda: linear(A, B, 1.0),
                lambda: linear_backward(None, A, B), lambda: rms_norm(A.double(), z(8)), lambda: rms_norm(A, None),
                lambda: rms_norm(A, z(8), eps="x"), lambda: rms_norm_backward(A, A, z(8), None)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(ValueError, match="CUDA"):
        rms_norm(A, z(8))
    with pytest.raises(ValueError, match="CUDA"):
        rms_norm_backward(A, A, z(8), torch.zeros(4))
