"""The root-mean-square norm with the residual's addition (include/wtconv_norm.h) on PyTorch tensors; the
marshalling is compiled (_binding).

``wtconv_rms_forward``, ``wtconv_rms_forward_e4m3`` and ``wtconv_rms_backward`` carry the C names and work on CUDA
tensors (..., C) whose rows are contiguous and lie at one distance from one another; ``rms_norm`` is
differentiable.  ``stream``, new tensors, their memory and graphs are as in ``scan`` and ``ssm``.
"""
from __future__ import annotations

import ctypes

import torch

from .ssm import _gradients, _rows
from .wtconv import load, load_binding

RMS_MAX_CHANNELS = 16384  # WTCONV_RMS_MAX_CHANNELS

EXPORTED = ("wtconv_rms_forward", "wtconv_rms_forward_e4m3", "wtconv_rms_workspace_size", "wtconv_rms_backward")


class RmsShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("rows", "C", "dtype", "total_dtype")] + [("eps", ctypes.c_float)]


class RmsTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("row", ctypes.c_longlong)]


_lib = _ext = None


def _load_ext():
    global _ext
    _ext = load_binding()
    return _ext


def _load() -> ctypes.CDLL:
    """The library with this header's signatures."""
    global _lib
    if _lib is None:
        lib = load()
        i, vp, sz, shape, tensor = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(RmsShape), ctypes.POINTER(RmsTensor)
        for name, result, arguments in (
                ("wtconv_rms_forward", i, [shape, tensor, tensor, vp, tensor, tensor, vp, vp]),
                ("wtconv_rms_forward_e4m3", i, [shape, tensor, tensor, vp, i, vp, vp, tensor, vp]),
                ("wtconv_rms_workspace_size", sz, [shape]),
                ("wtconv_rms_backward", i, [shape, tensor, tensor, vp, vp] + [tensor] * 3 + [vp, vp, sz, vp])):
            getattr(lib, name).restype = result
            getattr(lib, name).argtypes = arguments
        _lib = lib
    return _lib


def wtconv_rms_forward(x, weight, residual=None, eps=1e-6, y=None, total=None, stream=None):
    """(y, total, rstd): total = x + residual of the residual's dtype (x's or fp32; without a residual x itself),
    rstd = 1 / sqrt(mean total^2 + eps) fp32 for each row, y = total rstd weight of x's dtype.  weight (C,) fp32."""
    return (_ext or _load_ext()).rms_forward(x, weight, residual, eps, y, total, stream)


def wtconv_rms_forward_e4m3(x, weight, residual=None, eps=1e-6, block=0, total=None, stream=None):
    """(q, scales, total) with y = q scales: q in e4m3, scales fp32 (..., 1), or with ``block=128`` one for each 128
    neighbours (..., ceil(C / 128)); total is None without a residual."""
    return (_ext or _load_ext()).rms_forward_e4m3(x, weight, residual, eps, block, total, stream)


def wtconv_rms_backward(dy, total, weight, rstd, d_total=None, residual=True, workspace=None, stream=None):
    """(dx, d_residual, d_weight) from the forward's total and rstd; d_total is the gradient that flows into the total
    past the norm.  Of one dtype, dx and d_residual are one tensor; without a ``residual`` d_residual is None."""
    return (_ext or _load_ext()).rms_backward(dy, total, weight, rstd, d_total, residual, workspace, stream)


class WTConvRmsFunction(torch.autograd.Function):
    """Autograd wrapper: (y, total) through wtconv_rms_forward, gradients through wtconv_rms_backward; total is
    None without a residual.  A derivative of those gradients (``create_graph=True``) is refused."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, total, rstd = wtconv_rms_forward(x, weight, residual, eps)
        ctx.save_for_backward(total, weight, rstd)
        ctx.dtype, ctx.added = x.dtype, residual is not None
        ctx.set_materialize_grads(False)
        return y, None if residual is None else total

    @staticmethod
    def backward(ctx, dy, d_total):
        total, weight, rstd = ctx.saved_tensors
        dy = torch.zeros(total.shape, dtype=ctx.dtype, device=total.device) if dy is None else _rows(dy)

        def run():
            return wtconv_rms_backward(dy, total, weight, rstd, _rows(d_total), ctx.added)

        dx, d_residual, dw = _gradients("norm", run, total, weight, dy, d_total)
        return dx, dw, d_residual, None


def rms_norm(x, weight, residual=None, eps=1e-6):
    """Differentiable norm: y, or (y, total) with a residual; arguments as wtconv_rms_forward's.  First derivatives
    only."""
    y, total = WTConvRmsFunction.apply(x, weight, residual, eps)
    return y if residual is None else (y, total)
