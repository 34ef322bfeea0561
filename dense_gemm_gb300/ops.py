"""Python side of ``include/gemm_ops.h``: the product with its epilogue, the
root-mean-square norm, and their gradients.

The arguments are checked and marshalled by the extension ``_native`` (built
with the library); the arithmetic runs in the library's CUDA kernels. Outputs
and workspaces that are not given are allocated on the stream the kernels run
on (``stream``, or the current one); a workspace that is given is a contiguous
tensor of any type.

The calls record no gradient: outputs do not require one whatever the inputs do,
and ``linear_backward`` and ``rms_norm_backward`` are called by the caller's own
``torch.autograd.Function`` (``examples/mlp_block.py`` has both). C, ``pre``,
``residual``, ``grad`` and all matrices of the norms are stored by rows (unit
column stride, any row stride); A and B by rows or by columns, 8-bit ones with K
contiguous.
"""
import ctypes
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from .binding import GemmError, load_library

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
LINEAR_KERNELS = {"auto": 0, "pair": 1, "split": 2}

_ENTRIES = ("gemm_linear", "gemm_linear_workspace_size", "gemm_linear_backward", "gemm_linear_backward_workspace_size",
            "gemm_rms_norm", "gemm_rms_norm_backward", "gemm_rms_norm_backward_workspace_size")


class RmsNormResult(NamedTuple):
    """What ``rms_norm`` returns; ``h``, ``scale`` and ``rstd`` are None where they are not made."""
    y: torch.Tensor
    h: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


_module = None


def _native():
    """The marshalling extension, set up for the loaded library (once)."""
    global _module
    if _module is None:
        lib = load_library()
        from .build import native_path, native_unbuildable
        path = native_path()
        if not os.path.exists(path):
            raise GemmError(3, f"{path} is missing: {native_unbuildable() or 'build it with `python -m dense_gemm_gb300.build`'}")
        spec = importlib.util.spec_from_file_location(f"{__package__}._native", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.setup({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES}, GemmError, RmsNormResult)
        _module = module
    return _module


def _code(table: dict, key, what: str) -> int:
    code = table.get(key)
    if code is None:
        raise ValueError(f"{what} must be one of {list(table)}, got {key!r}")
    return code


def linear_workspace_size(A: torch.Tensor, B: torch.Tensor) -> int:
    """Workspace bytes of ``linear`` for these operands: 0 where their bases and
    row strides are multiples of 16 bytes."""
    return _native().linear_workspace_size(A, B)


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
    return (_module or _native()).linear(
        A, B, bias, _code(ACTIVATIONS, activation, "activation"), residual, scale_a, scale_b, out, out_dtype, pre,
        bool(return_pre), _code(LINEAR_KERNELS, kernel, "kernel"), workspace, stream)


def linear_backward(grad: torch.Tensor, A: torch.Tensor, B: torch.Tensor, *, pre: torch.Tensor = None,
                    activation: str = "none", need_a: bool = True, need_b: bool = True, need_bias: bool = False,
                    grad_dtype: torch.dtype = None, kernel: str = "auto", workspace: torch.Tensor = None, stream=None):
    """(dA, dB, dbias) of ``linear`` (16-bit operands, no scales) from ``grad``
    [M, N], the gradient of C, in A's type; None for what is not needed.

    ``pre`` is what ``linear(..., return_pre=True)`` kept (needed with an
    activation). dA [M, K] and dB [K, N] have ``grad_dtype`` (default A's type)
    and the memory order of A and B; dbias [N] is float32. The residual's
    gradient is ``grad`` itself. With an activation, D = grad * act'(pre) is
    rounded to A's type for the two products, whatever ``grad_dtype`` is; dbias is
    summed from D before that.
    """
    return (_module or _native()).linear_backward(
        grad, A, B, pre, _code(ACTIVATIONS, activation, "activation"), bool(need_a), bool(need_b), bool(need_bias), grad_dtype,
        _code(LINEAR_KERNELS, kernel, "kernel"), workspace, stream)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: torch.Tensor = None, eps: float = 1e-6,
             out_dtype: torch.dtype = None, return_rstd: bool = False, out: torch.Tensor = None,
             h_out: torch.Tensor = None, stream=None) -> RmsNormResult:
    """h = x + residual; y = weight * h / sqrt(mean(h^2) + eps), row by row.

    x [rows, width] is float32, float16 or bfloat16; ``weight`` [width] has x's
    type or is float32. y has x's type, or with ``out_dtype=torch.float8_e4m3fn``
    holds 8-bit floats whose value is y * scale[:, None] (``scale`` fp32
    [rows]): an A and scale_a for ``linear``; rows of zeros, and rows whose largest
    |y| is below 7.7e-34, are zeros with scale 1. ``h`` (x's type) is made when a
    residual is given; ``h_out`` may be x or residual itself. ``return_rstd``
    keeps 1 / sqrt(mean(h^2) + eps) for ``rms_norm_backward``.
    """
    return (_module or _native()).rms_norm(x, weight, residual, eps, out_dtype, bool(return_rstd), out, h_out, stream)


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
    return (_module or _native()).rms_norm_backward(grad, h, weight, rstd, grad_h, bool(need_weight), out, workspace, stream)
