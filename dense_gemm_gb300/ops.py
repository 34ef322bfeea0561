"""ctypes binding of ``include/gemm_ops.h`` (argument marshalling only): the
product with its epilogue, the root-mean-square norm, and their gradients.

Outputs and workspaces that are not given are allocated on the stream the
kernels run on (``stream``, or the current one).
"""
import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import GemmError, _check, load_library  # noqa: F401

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LINEAR_KERNELS = {"auto": 0, "pair": 1, "split": 2}

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}
_C_TYPES = (torch.float32, torch.float16, torch.bfloat16)
_OPERANDS = (torch.float16, torch.bfloat16, torch.float8_e4m3fn)


class _Matrix(ctypes.Structure):  # gemm_matrix_t
    _fields_ = [("data", ctypes.c_void_p), ("stride_row", ctypes.c_int64), ("stride_col", ctypes.c_int64),
                ("type", ctypes.c_int32)]


class _Epilogue(ctypes.Structure):  # gemm_epilogue_t
    _fields_ = [("bias", ctypes.c_void_p), ("bias_type", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("scale_a", ctypes.c_void_p), ("scale_b", ctypes.c_void_p), ("residual", _Matrix), ("pre", _Matrix)]


_ready = None


def _lib():
    global _ready
    if _ready is not None:
        return _ready
    lib = load_library()
    m, e, vp = ctypes.POINTER(_Matrix), ctypes.POINTER(_Epilogue), ctypes.c_void_p
    i64, i32, u32, u64, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float
    pu64 = ctypes.POINTER(u64)
    lib.gemm_linear.argtypes = [m, m, m, e, i64, i64, i64, u32, vp, u64, vp]
    lib.gemm_linear_workspace_size.argtypes = [m, m, i64, i64, i64, pu64]
    lib.gemm_linear_backward.argtypes = [m, m, m, m, i32, m, m, vp, i64, i64, i64, u32, vp, u64, vp]
    lib.gemm_linear_backward_workspace_size.argtypes = [m, m, m, i32, i32, i64, i64, i64, pu64]
    lib.gemm_rms_norm.argtypes = [m, m, vp, i32, m, m, vp, vp, i64, i64, f32, vp]
    lib.gemm_rms_norm_backward.argtypes = [m, m, vp, i32, vp, m, m, vp, i64, i64, vp, u64, vp]
    lib.gemm_rms_norm_backward_workspace_size.argtypes = [i64, i64, pu64]
    for name in ("gemm_linear", "gemm_linear_workspace_size", "gemm_linear_backward",
                 "gemm_linear_backward_workspace_size", "gemm_rms_norm", "gemm_rms_norm_backward",
                 "gemm_rms_norm_backward_workspace_size"):
        getattr(lib, name).restype = ctypes.c_int
    _ready = lib
    return lib


def _matrix(t: Optional[torch.Tensor]) -> _Matrix:
    """The tensor's gemm_matrix_t. torch gives dimensions of one element any
    stride, also 0; a stride of 0 elsewhere (an expanded tensor) goes through
    and is refused."""
    if t is None:
        return _Matrix(None, 1, 1, 0)
    r, c = t.stride()
    rows, cols = t.shape
    return _Matrix(t.data_ptr(), r if r or rows > 1 else 1, c if c or cols > 1 else 1, _TYPES[t.dtype])


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@contextlib.contextmanager
def _other_device(dev):
    with torch.cuda.device(dev):
        yield


class _Here:
    """Stands in for the device and stream contexts where nothing changes."""

    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


_HERE = _Here()


def _on(dev: torch.device, stream):
    """(contexts' handle, device context, allocation context): the C entry points
    act on the current device, and new tensors belong to the stream they are
    written on."""
    device = _HERE if torch.cuda.current_device() == dev.index else _other_device(dev)
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream, device, _HERE
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return stream.cuda_stream, device, torch.cuda.stream(stream)


def _one_device(first: torch.Tensor, *others) -> torch.device:
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("the operators take CUDA tensors")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"all tensors must be on one CUDA device, got {dev} and {t.device}")
    return dev


def _matrix_like(t, shape, dtype, what):
    if t is not None and (tuple(t.shape) != shape or t.dtype != dtype):
        raise ValueError(f"{what} must be {dtype} of shape {list(shape)}, got {t.dtype} {list(t.shape)}")


def _vector(t, n, dtypes, what):
    if t is None:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be one of {dtypes}, got {t.dtype}")
    if tuple(t.shape) != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous vector of {n} elements, got shape {list(t.shape)}")


def _workspace(given, need, dev, what):
    """(tensor, bytes): the caller's workspace, or one of `need` bytes."""
    if given is None:
        given = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        return given, need
    if given.device != dev:
        raise ValueError(f"{what}: the workspace is on {given.device}, the tensors on {dev}")
    return given, given.numel() * given.element_size()


def _operands(A, B):
    if A.dtype not in _OPERANDS or A.dtype != B.dtype:
        raise TypeError(f"A and B must both be float16, bfloat16 or float8_e4m3fn, got {A.dtype} and {B.dtype}")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shapes {tuple(A.shape)} @ {tuple(B.shape)} do not chain")


def linear_workspace_size(A: torch.Tensor, B: torch.Tensor) -> int:
    """Workspace bytes of ``linear`` for these operands: 0 where their bases and
    row strides are multiples of 16 bytes."""
    _operands(A, B)
    n = ctypes.c_uint64()
    _check(_lib().gemm_linear_workspace_size(_matrix(A), _matrix(B), A.shape[0], B.shape[1], A.shape[1], n),
           "gemm_linear_workspace_size")
    return int(n.value)


def linear(A: torch.Tensor, B: torch.Tensor, bias: torch.Tensor = None, *, activation: str = "none",
           residual: torch.Tensor = None, scale_a: torch.Tensor = None, scale_b: torch.Tensor = None,
           out: torch.Tensor = None, out_dtype: torch.dtype = None, pre: torch.Tensor = None,
           return_pre: bool = False, kernel: str = "auto", workspace: torch.Tensor = None, stream=None):
    """C = act(scale_a[:, None] * scale_b * (A @ B) + bias) + residual.

    A [M, K] and B [K, N] are float16, bfloat16, or float8_e4m3fn with fp32
    ``scale_a`` [M] and ``scale_b`` [N]; a weight kept as [N, K] goes in as its
    transpose. ``activation``: "none", "relu", "gelu", "gelu_tanh" or "silu".
    C has ``out``'s type or ``out_dtype``, else the residual's, else A's
    (bfloat16 for 8-bit operands); ``residual`` [M, N] has C's type and may be
    ``out`` itself; ``bias`` [N] has C's type or is float32. With ``return_pre``
    (or a ``pre`` [M, N] to write) the value before the activation is kept, and
    (C, pre) is returned. ``kernel`` chooses between "pair" and "split" by hand
    (gemm_linear in include/gemm_ops.h).
    """
    _operands(A, B)
    (M, K), N = A.shape, B.shape[1]
    eight = A.dtype == torch.float8_e4m3fn
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    if kernel not in LINEAR_KERNELS:
        raise ValueError(f"kernel must be one of {list(LINEAR_KERNELS)}, got {kernel!r}")
    if eight != (scale_a is not None) or eight != (scale_b is not None):
        raise ValueError("scale_a and scale_b go with float8_e4m3fn operands, and only with them")
    dtype = out.dtype if out is not None else out_dtype if out_dtype is not None else residual.dtype \
        if residual is not None else torch.bfloat16 if eight else A.dtype
    if dtype not in _C_TYPES:
        raise TypeError(f"C must be float32, float16 or bfloat16, got {dtype}")
    dev = _one_device(A, B, bias, residual, scale_a, scale_b, out, pre)
    _matrix_like(out, (M, N), dtype, "out")
    _matrix_like(residual, (M, N), dtype, "residual")
    _matrix_like(pre, (M, N), dtype, "pre")
    _vector(bias, N, (torch.float32, dtype), "bias")
    _vector(scale_a, M, (torch.float32,), "scale_a")
    _vector(scale_b, N, (torch.float32,), "scale_b")
    lib = _lib()
    handle, device, alloc = _on(dev, stream)
    a, b = _matrix(A), _matrix(B)
    need = ctypes.c_uint64()
    _check(lib.gemm_linear_workspace_size(a, b, M, N, K, need), "gemm_linear")
    with device, alloc:
        if out is None:
            out = torch.empty((M, N), dtype=dtype, device=dev)
        if pre is None and return_pre:
            pre = torch.empty((M, N), dtype=dtype, device=dev)
        ws, ws_bytes = _workspace(workspace, need.value, dev, "linear")
        ep = _Epilogue(_ptr(bias), _TYPES[bias.dtype] if bias is not None else 0, ACTIVATIONS[activation], _ptr(scale_a),
                       _ptr(scale_b), _matrix(residual), _matrix(pre))
        _check(lib.gemm_linear(a, b, _matrix(out), ep, M, N, K, LINEAR_KERNELS[kernel], _ptr(ws), ws_bytes, handle),
               "gemm_linear")
    return (out, pre) if pre is not None else out


def _empty_like_order(t, dtype):
    """A new matrix of t's shape, stored by columns where t is (a weight kept as [N, K])."""
    (r, c), by_columns = t.shape, t.stride(0) == 1 and t.stride(1) != 1
    return torch.empty((c, r), dtype=dtype, device=t.device).t() if by_columns else \
        torch.empty((r, c), dtype=dtype, device=t.device)


def linear_backward(grad: torch.Tensor, A: torch.Tensor, B: torch.Tensor, *, pre: torch.Tensor = None,
                    activation: str = "none", need_a: bool = True, need_b: bool = True, need_bias: bool = False,
                    grad_dtype: torch.dtype = None, kernel: str = "auto", workspace: torch.Tensor = None, stream=None):
    """(dA, dB, dbias) of ``linear`` (16-bit operands, no scales) from ``grad``
    [M, N], the gradient of C, in A's type; None for what is not needed.

    ``pre`` is what ``linear(..., return_pre=True)`` kept (needed with an
    activation). dA [M, K] and dB [K, N] have ``grad_dtype`` (default A's type)
    and the memory order of A and B; dbias [N] is float32. The residual's
    gradient is ``grad`` itself.
    """
    _operands(A, B)
    if A.dtype == torch.float8_e4m3fn:
        raise TypeError("linear_backward takes float16 or bfloat16 operands")
    (M, K), N = A.shape, B.shape[1]
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, got {activation!r}")
    if kernel not in LINEAR_KERNELS:
        raise ValueError(f"kernel must be one of {list(LINEAR_KERNELS)}, got {kernel!r}")
    if activation != "none" and pre is None:
        raise ValueError("with an activation, linear_backward needs pre (linear(..., return_pre=True))")
    if activation == "none":
        pre = None
    dtype = A.dtype if grad_dtype is None else grad_dtype
    if dtype not in _C_TYPES:
        raise TypeError(f"gradients are float32, float16 or bfloat16, got {dtype}")
    dev = _one_device(grad, A, B, pre)
    _matrix_like(grad, (M, N), A.dtype, "grad")
    _matrix_like(pre, (M, N), A.dtype, "pre")
    lib = _lib()
    handle, device, alloc = _on(dev, stream)
    g, a, b = _matrix(grad), _matrix(A), _matrix(B)
    act = ACTIVATIONS[activation]
    need = ctypes.c_uint64()
    _check(lib.gemm_linear_backward_workspace_size(g, a, b, act, int(need_bias), M, N, K, need), "gemm_linear_backward")
    with device, alloc:
        dA = _empty_like_order(A, dtype) if need_a else None
        dB = _empty_like_order(B, dtype) if need_b else None
        dbias = torch.empty(N, dtype=torch.float32, device=dev) if need_bias else None
        ws, ws_bytes = _workspace(workspace, need.value, dev, "linear_backward")
        _check(lib.gemm_linear_backward(g, a, b, _matrix(pre), act, _matrix(dA), _matrix(dB), _ptr(dbias), M, N, K,
                                        LINEAR_KERNELS[kernel], _ptr(ws), ws_bytes, handle), "gemm_linear_backward")
    return dA, dB, dbias


class RmsNormResult(NamedTuple):
    """What ``rms_norm`` returns; ``h``, ``scale`` and ``rstd`` are None where they are not made."""
    y: torch.Tensor
    h: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor = None, eps: float = 1e-6,
             out_dtype: torch.dtype = None, return_rstd: bool = False, out: torch.Tensor = None,
             h_out: torch.Tensor = None, stream=None) -> RmsNormResult:
    """h = x + residual; y = weight * h / sqrt(mean(h^2) + eps), row by row.

    x [rows, width] is float32, float16 or bfloat16; ``weight`` [width] has x's
    type or is float32. y has x's type, or with ``out_dtype=torch.float8_e4m3fn``
    holds 8-bit floats whose value is y * scale[:, None] (``scale`` fp32
    [rows]): an A and scale_a for ``linear``. ``h`` (x's type) is made when a
    residual is given; ``h_out`` may be x or residual itself. ``return_rstd``
    keeps 1 / sqrt(mean(h^2) + eps) for ``rms_norm_backward``.
    """
    if x.dim() != 2 or x.dtype not in _C_TYPES:
        raise TypeError(f"x must be a float32, float16 or bfloat16 matrix, got {x.dtype} {list(x.shape)}")
    rows, width = x.shape
    dtype = out.dtype if out is not None else x.dtype if out_dtype is None else out_dtype
    if dtype not in (x.dtype, torch.float8_e4m3fn):
        raise TypeError(f"y has x's type or float8_e4m3fn, got {dtype}")
    dev = _one_device(x, weight, residual, out, h_out)
    _vector(weight, width, (torch.float32, x.dtype), "weight")
    _matrix_like(residual, (rows, width), x.dtype, "residual")
    _matrix_like(out, (rows, width), dtype, "out")
    _matrix_like(h_out, (rows, width), x.dtype, "h_out")
    if h_out is not None and residual is None:
        raise ValueError("h_out goes with a residual: without one h is x")
    lib = _lib()
    handle, device, alloc = _on(dev, stream)
    with device, alloc:
        y = out if out is not None else torch.empty((rows, width), dtype=dtype, device=dev)
        h = None if residual is None else h_out if h_out is not None else \
            torch.empty((rows, width), dtype=x.dtype, device=dev)
        scale = torch.empty(rows, dtype=torch.float32, device=dev) if dtype == torch.float8_e4m3fn else None
        rstd = torch.empty(rows, dtype=torch.float32, device=dev) if return_rstd else None
        _check(lib.gemm_rms_norm(_matrix(x), _matrix(residual), weight.data_ptr(), _TYPES[weight.dtype], _matrix(y),
                                 _matrix(h), _ptr(scale), _ptr(rstd), rows, width, eps, handle), "gemm_rms_norm")
    return RmsNormResult(y, h, scale, rstd)


def rms_norm_backward(grad: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                      grad_h: torch.Tensor = None, need_weight: bool = True, out: torch.Tensor = None,
                      workspace: torch.Tensor = None, stream=None):
    """(dx, dweight) of ``rms_norm`` from ``grad``, the gradient of y, and
    ``grad_h``, the gradient that arrives at h on the residual path.

    ``h`` is the forward call's h (x where there was no residual) and ``rstd``
    what ``return_rstd=True`` kept. dx is the gradient of x and of the residual;
    ``out`` may be grad or grad_h itself. dweight is float32 [width], None
    unless ``need_weight``.
    """
    if h.dim() != 2 or h.dtype not in _C_TYPES:
        raise TypeError(f"h must be a float32, float16 or bfloat16 matrix, got {h.dtype} {list(h.shape)}")
    rows, width = h.shape
    dev = _one_device(h, grad, weight, rstd, grad_h, out)
    _matrix_like(grad, (rows, width), h.dtype, "grad")
    _matrix_like(grad_h, (rows, width), h.dtype, "grad_h")
    _matrix_like(out, (rows, width), h.dtype, "out")
    _vector(weight, width, (torch.float32, h.dtype), "weight")
    _vector(rstd, rows, (torch.float32,), "rstd")
    lib = _lib()
    handle, device, alloc = _on(dev, stream)
    need = ctypes.c_uint64()
    if need_weight:
        _check(lib.gemm_rms_norm_backward_workspace_size(rows, width, need), "gemm_rms_norm_backward")
    with device, alloc:
        dx = out if out is not None else torch.empty((rows, width), dtype=h.dtype, device=dev)
        dweight = torch.empty(width, dtype=torch.float32, device=dev) if need_weight else None
        ws, ws_bytes = _workspace(workspace, need.value, dev, "rms_norm_backward")
        _check(lib.gemm_rms_norm_backward(_matrix(grad), _matrix(h), weight.data_ptr(), _TYPES[weight.dtype], _ptr(rstd),
                                          _matrix(grad_h), _matrix(dx), _ptr(dweight), rows, width, _ptr(ws), ws_bytes,
                                          handle), "gemm_rms_norm_backward")
    return dx, dweight
