"""The gated scan (include/wtconv_scan.h) on PyTorch tensors; the marshalling is compiled (_binding).

``wtconv_scan_forward``, ``wtconv_scan_backward`` and ``wtconv_scan_step`` carry the C names and
work on CUDA tensors; ``WTConvScanFunction`` (and ``gated_scan`` around it) makes the scan
differentiable.  Activations are planes (B, C, T) or (B, C, H, W) with ``layout="planes"``, or
tokens (B, T, C) with ``layout="tokens"``; the innermost axis must be contiguous, the others may
have any strides (one half of a projection's output, a slice of a batch).

``stream`` (default: the current one) is where a call's work is queued, and new tensors are allocated
for it.  The caller orders it after the work that makes the inputs and before what reads the outputs;
memory of a tensor that is let go of meanwhile is not used again before the work has ended, except with
an ``ExternalStream``, whose owner keeps the tensors.
"""
from __future__ import annotations

import ctypes

import torch

from .wtconv import _raise, _stream, load, load_binding

SCAN_KEEP = 64  # WTCONV_SCAN_KEEP
OP_SCAN_FORWARD, OP_SCAN_BACKWARD = 0, 1

EXPORTED = ("wtconv_scan_workspace_size", "wtconv_scan_status", "wtconv_scan_selftest_wait_timeout", "wtconv_scan_forward",
            "wtconv_scan_backward", "wtconv_scan_step")

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
        i, q, vp, sz = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t
        act = [vp, q, q]
        lib.wtconv_scan_workspace_size.restype = sz
        lib.wtconv_scan_workspace_size.argtypes = [i] * 6
        lib.wtconv_scan_status.restype = i
        lib.wtconv_scan_status.argtypes = []
        lib.wtconv_scan_selftest_wait_timeout.restype = i
        lib.wtconv_scan_selftest_wait_timeout.argtypes = [vp]
        lib.wtconv_scan_forward.restype = i
        lib.wtconv_scan_forward.argtypes = [i] * 5 + act * 2 + [vp] * 3 + act + [vp, vp, vp, sz, vp]
        lib.wtconv_scan_backward.restype = i
        lib.wtconv_scan_backward.argtypes = [i] * 5 + act * 2 + [vp] * 3 + act + [vp] + act * 2 + [vp, vp, vp, sz, vp]
        lib.wtconv_scan_step.restype = i
        lib.wtconv_scan_step.argtypes = [i] * 3 + [vp, q] * 2 + [vp, vp, i, vp, vp, q, vp]
        _lib = lib
    return _lib


def wtconv_scan_workspace_size(op: int, B: int, T: int, C: int, layout: int, dtype: int) -> int:
    return _load().wtconv_scan_workspace_size(op, B, T, C, layout, dtype)


def wtconv_scan_status() -> int:
    """Synchronise the device; wtconv.ERR_DEVICE_TIMEOUT if a scan's bounded wait gave up."""
    return _load().wtconv_scan_status()


def wtconv_scan_selftest_wait_timeout(stream=None) -> None:
    """Launch the diagnostic whose one bounded wait is never completed: the next
    wtconv_scan_status() then returns wtconv.ERR_DEVICE_TIMEOUT."""
    _raise(_load().wtconv_scan_selftest_wait_timeout(_stream(stream)), "wtconv_scan_selftest_wait_timeout")


def wtconv_scan_forward(x, gate, gate_bias, h0=None, lengths=None, layout="planes", keep_states=False, y=None,
                        workspace=None, stream=None):
    """(y, h_last, states) of h_t = a_t h_{t-1} + (1 - a_t) x_t, a = sigmoid(gate + gate_bias).

    gate_bias (C,) and h0 (B, C) fp32; lengths (B,) int32 ends each sequence.  ``states`` is what
    the backward needs (None unless ``keep_states``); h_last (B, C) fp32 is the state after each
    sequence's last position."""
    return (_ext or _load_ext()).scan_forward(x, gate, gate_bias, h0, lengths, layout, keep_states, y, workspace, stream)


def wtconv_scan_backward(x, gate, gate_bias, states, dy, dh_last=None, lengths=None, layout="planes", dx=None,
                         d_gate=None, workspace=None, stream=None):
    """(dx, d_gate, d_gate_bias, d_h0) from the forward's inputs and its ``states``."""
    return (_ext or _load_ext()).scan_backward(x, gate, gate_bias, states, dy, dh_last, lengths, layout, dx, d_gate,
                                               workspace, stream)


def wtconv_scan_step(x, gate, gate_bias, pool, slots=None, y=None, stream=None):
    """One position of B sequences: x, gate (B, C); updates rows of ``pool`` (n_states, C) fp32 in
    place and returns y (B, C).  Sequence b owns row slots[b] (int32; row b without slots); a slot
    outside the pool marks an idle sequence, whose y is 0."""
    return (_ext or _load_ext()).scan_step(x, gate, gate_bias, pool, slots, y, stream)


class _ScanGradients(torch.autograd.Function):
    """wtconv_scan_backward as an operation of its own, so that a second derivative meets its refusal."""

    @staticmethod
    def forward(ctx, x, gate, gate_bias, h0, states, dy, dh_last, lengths, layout):
        ctx.set_materialize_grads(False)
        return wtconv_scan_backward(x, gate, gate_bias, states, dy, dh_last, lengths, layout)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the gated scan has no second derivative")


class WTConvScanFunction(torch.autograd.Function):
    """Autograd wrapper: (y, h_last) through wtconv_scan_forward, gradients through wtconv_scan_backward.
    A derivative of those gradients (``create_graph=True``) is refused."""

    @staticmethod
    def forward(ctx, x, gate, gate_bias, h0, lengths, layout):
        y, h_last, states = wtconv_scan_forward(x, gate, gate_bias, h0, lengths, layout,
                                                keep_states=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, gate, gate_bias, states, lengths)
        ctx.layout = layout
        ctx.h0 = h0  # for its place in the graph only: the backward does not read its values, which may change
        ctx.set_materialize_grads(False)
        return y, h_last

    @staticmethod
    def backward(ctx, dy, dh_last):
        x, gate, gate_bias, states, lengths = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dh_last = None if dh_last is None else dh_last.contiguous()
        if torch.is_grad_enabled():  # create_graph=True
            grads = _ScanGradients.apply(x, gate, gate_bias, ctx.h0, states, dy, dh_last, lengths, ctx.layout)
        else:
            grads = wtconv_scan_backward(x, gate, gate_bias, states, dy, dh_last, lengths, ctx.layout)
        dx, d_gate, d_bias, d_h0 = grads
        return dx, d_gate, d_bias, None if ctx.h0 is None else d_h0, None, None


def gated_scan(x, gate, gate_bias, h0=None, lengths=None, layout="planes"):
    """Differentiable gated scan: (y, h_last); arguments as wtconv_scan_forward's.  First derivatives only."""
    return WTConvScanFunction.apply(x, gate, gate_bias, h0, lengths, layout)
