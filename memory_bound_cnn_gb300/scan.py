"""Python binding of the gated scan (include/wtconv_scan.h): argument marshalling only.

``wtconv_scan_forward``, ``wtconv_scan_backward`` and ``wtconv_scan_step`` carry the C names and
work on CUDA tensors; ``WTConvScanFunction`` (and ``gated_scan`` around it) makes the scan
differentiable.  Activations are planes (B, C, T) or (B, C, H, W) with ``layout="planes"``, or
tokens (B, T, C) with ``layout="tokens"``; the innermost axis must be contiguous, the others may
have any strides (one half of a projection's output, a slice of a batch).
"""
from __future__ import annotations

import ctypes

import torch

from .wtconv import DTYPE_CODE, _on, _ptr, _raise, _stream, load

LAYOUTS = {"planes": 0, "tokens": 1}
SCAN_KEEP = 64  # WTCONV_SCAN_KEEP
OP_SCAN_FORWARD, OP_SCAN_BACKWARD = 0, 1

EXPORTED = ("wtconv_scan_workspace_size", "wtconv_scan_forward", "wtconv_scan_backward", "wtconv_scan_step")

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = load()
        i, q, vp, sz = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_size_t
        act = [vp, q, q]
        lib.wtconv_scan_workspace_size.restype = sz
        lib.wtconv_scan_workspace_size.argtypes = [i] * 6
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


def _act(t: torch.Tensor, name: str, layout: str, like: torch.Tensor | None = None) -> torch.Tensor:
    """The activation as a 3-D tensor with a contiguous innermost axis."""
    if not t.is_cuda or t.dtype not in DTYPE_CODE:
        raise ValueError(f"{name} must be a CUDA tensor of fp32, bf16 or fp16, not {t.dtype} on {t.device}")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must match x's shape, dtype and device")
    if t.dim() == 4 and layout == "planes":
        B, C, H, W = t.shape
        if t.stride(3) != 1 and W > 1 or t.stride(2) != W and H > 1:
            raise ValueError(f"{name}: the pixels of a plane must be contiguous")
        t = t.as_strided((B, C, H * W), (t.stride(0), t.stride(1), 1))
    if t.dim() != 3:
        raise ValueError(f"{name} must be (B, C, T) or (B, C, H, W) planes, or (B, T, C) tokens")
    if t.numel() == 0:
        raise ValueError(f"{name} is empty")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the innermost axis must be contiguous")
    return t


def _f32(t: torch.Tensor | None, name: str, shape: tuple, device, dtype=torch.float32):
    if t is None:
        return None
    if t.device != device or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")
    return _ptr(t)


def _dims(x3: torch.Tensor, layout: str):
    B, C, T = x3.shape if layout == "planes" else (x3.shape[0], x3.shape[2], x3.shape[1])
    return B, T, C, LAYOUTS[layout], DTYPE_CODE[x3.dtype]


def _view(t: torch.Tensor):
    return _ptr(t), t.stride(0), t.stride(1)


def _scratch(op: int, dims, device, workspace):
    need = _load().wtconv_scan_workspace_size(op, *dims)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def _check_layout(layout: str):
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be 'planes' or 'tokens', not {layout!r}")


def wtconv_scan_forward(x, gate, gate_bias, h0=None, lengths=None, layout="planes", keep_states=False, y=None,
                        workspace=None, stream=None):
    """(y, h_last, states) of h_t = a_t h_{t-1} + (1 - a_t) x_t, a = sigmoid(gate + gate_bias).

    gate_bias (C,) and h0 (B, C) fp32; lengths (B,) int32 ends each sequence.  ``states`` is what
    the backward needs (None unless ``keep_states``); h_last (B, C) fp32 is the state after each
    sequence's last position."""
    _check_layout(layout)
    x3, g3 = _act(x, "x", layout), _act(gate, "gate", layout, x)
    dims = B, T, C, _, _ = _dims(x3, layout)
    dev = x.device
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    y3 = _act(y, "y", layout, x)
    bias_p, h0_p = _f32(gate_bias, "gate_bias", (C,), dev), _f32(h0, "h0", (B, C), dev)
    len_p = _f32(lengths, "lengths", (B,), dev, torch.int32)
    h_last = torch.empty((B, C), dtype=torch.float32, device=dev)
    n = -(-T // SCAN_KEEP)
    states = None
    if keep_states:
        states = torch.empty((B, C, n) if layout == "planes" else (B, n, C), dtype=torch.float32, device=dev)
    with _on(dev, stream, workspace):
        ws, nbytes = _scratch(OP_SCAN_FORWARD, dims, dev, workspace)
        rc = _load().wtconv_scan_forward(*dims, *_view(x3), *_view(g3), bias_p, h0_p, len_p, *_view(y3), _ptr(h_last),
                                         _ptr(states), _ptr(ws), nbytes, _stream(stream))
    _raise(rc, "wtconv_scan_forward")
    return y, h_last, states


def wtconv_scan_backward(x, gate, gate_bias, states, dy, dh_last=None, lengths=None, layout="planes", dx=None,
                         d_gate=None, workspace=None, stream=None):
    """(dx, d_gate, d_gate_bias, d_h0) from the forward's inputs and its ``states``."""
    _check_layout(layout)
    x3, g3, dy3 = _act(x, "x", layout), _act(gate, "gate", layout, x), _act(dy, "dy", layout, x)
    dims = B, T, C, _, _ = _dims(x3, layout)
    dev = x.device
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev) if dx is None else dx
    d_gate = torch.empty(x.shape, dtype=x.dtype, device=dev) if d_gate is None else d_gate
    dx3, dg3 = _act(dx, "dx", layout, x), _act(d_gate, "d_gate", layout, x)
    n = -(-T // SCAN_KEEP)
    bias_p = _f32(gate_bias, "gate_bias", (C,), dev)
    if states is None:
        raise ValueError("the backward needs the states of a forward with keep_states=True")
    st_p = _f32(states, "states", (B, C, n) if layout == "planes" else (B, n, C), dev)
    dh_p = _f32(dh_last, "dh_last", (B, C), dev)
    len_p = _f32(lengths, "lengths", (B,), dev, torch.int32)
    d_bias = torch.empty((C,), dtype=torch.float32, device=dev)
    d_h0 = torch.empty((B, C), dtype=torch.float32, device=dev)
    with _on(dev, stream, workspace):
        ws, nbytes = _scratch(OP_SCAN_BACKWARD, dims, dev, workspace)
        rc = _load().wtconv_scan_backward(*dims, *_view(x3), *_view(g3), bias_p, st_p, len_p, *_view(dy3), dh_p,
                                          *_view(dx3), *_view(dg3), _ptr(d_bias), _ptr(d_h0), _ptr(ws), nbytes,
                                          _stream(stream))
    _raise(rc, "wtconv_scan_backward")
    return dx, d_gate, d_bias, d_h0


def wtconv_scan_step(x, gate, gate_bias, pool, slots=None, y=None, stream=None):
    """One position of B sequences: x, gate (B, C); updates rows of ``pool`` (n_states, C) fp32 in
    place and returns y (B, C).  Sequence b owns row slots[b] (int32; row b without slots); a slot
    outside the pool marks an idle sequence, whose y is 0."""
    if x.dim() != 2 or x.numel() == 0 or not x.is_cuda or x.dtype not in DTYPE_CODE:
        raise ValueError("x must be a non-empty (B, C) CUDA tensor of fp32, bf16 or fp16")
    B, C = x.shape
    dev = x.device
    if y is None:
        y = torch.empty((B, C), dtype=x.dtype, device=dev)
    for t, name in ((x, "x"), (gate, "gate"), (y, "y")):
        if t.shape != x.shape or t.dtype != x.dtype or t.device != dev or (t.stride(1) != 1 and C > 1):
            raise ValueError(f"{name} must match x's shape, dtype and device and be contiguous along C")
    if pool.dim() != 2 or pool.shape[1] != C or pool.shape[0] < 1:
        raise ValueError(f"pool must be (n_states, {C})")
    bias_p, pool_p = _f32(gate_bias, "gate_bias", (C,), dev), _f32(pool, "pool", tuple(pool.shape), dev)
    slots_p = _f32(slots, "slots", (B,), dev, torch.int32)
    with _on(dev, stream, None):
        rc = _load().wtconv_scan_step(B, C, DTYPE_CODE[x.dtype], _ptr(x), x.stride(0), _ptr(gate), gate.stride(0),
                                      bias_p, pool_p, pool.shape[0], slots_p, _ptr(y), y.stride(0), _stream(stream))
    _raise(rc, "wtconv_scan_step")
    return y


class WTConvScanFunction(torch.autograd.Function):
    """Autograd wrapper: (y, h_last) through wtconv_scan_forward, gradients through wtconv_scan_backward."""

    @staticmethod
    def forward(ctx, x, gate, gate_bias, h0, lengths, layout):
        y, h_last, states = wtconv_scan_forward(x, gate, gate_bias, h0, lengths, layout, keep_states=True)
        ctx.save_for_backward(x, gate, gate_bias, states, lengths)
        ctx.layout, ctx.has_h0 = layout, h0 is not None
        ctx.set_materialize_grads(False)
        return y, h_last

    @staticmethod
    def backward(ctx, dy, dh_last):
        x, gate, gate_bias, states, lengths = ctx.saved_tensors
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else dy.contiguous()
        dh_last = None if dh_last is None else dh_last.contiguous()
        dx, d_gate, d_bias, d_h0 = wtconv_scan_backward(x, gate, gate_bias, states, dy, dh_last, lengths, ctx.layout)
        return dx, d_gate, d_bias, d_h0 if ctx.has_h0 else None, None, None


def gated_scan(x, gate, gate_bias, h0=None, lengths=None, layout="planes"):
    """Differentiable gated scan: (y, h_last); arguments as wtconv_scan_forward's."""
    return WTConvScanFunction.apply(x, gate, gate_bias, h0, lengths, layout)
