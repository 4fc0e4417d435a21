"""The selective state space scan and the short causal convolution (include/wtconv_ssm.h) on PyTorch tensors;
the marshalling is compiled (_binding).

``wtconv_selective_forward``, ``_backward`` and ``_step`` and ``wtconv_causal_forward``, ``_backward`` and
``_step`` carry the C names and work on CUDA tensors; ``selective_scan`` and ``causal_conv`` are differentiable.
Activations are planes (B, C, T) or (B, C, H, W) with ``layout="planes"``, or tokens (B, T, C) with
``layout="tokens"``, as for the gated scan; what a position writes to the states and reads from them, ``B`` and ``C``,
is (B, G, N, T) or (B, G, N, H, W), or (B, T, G, N).  The innermost axis must be contiguous, and G and N must follow
one another; the others may have any strides.

``stream``, new tensors and their memory are as in ``scan``.  The calls can be captured in a CUDA graph, the
functions that carry the C names forward and backward alike.  A ``backward()`` of autograd is captured on leaves that no
eager graph still holds (PyTorch ends the process otherwise).
"""
from __future__ import annotations

import ctypes

import torch

from .scan import _recorded
from .wtconv import load, load_binding

SELECTIVE_KEEP = 16        # WTCONV_SELECTIVE_KEEP
SELECTIVE_MAX_STATES = 64  # WTCONV_SELECTIVE_MAX_STATES

EXPORTED = ("wtconv_selective_states_size", "wtconv_selective_workspace_size", "wtconv_selective_forward",
            "wtconv_selective_backward", "wtconv_selective_step", "wtconv_causal_workspace_size", "wtconv_causal_forward",
            "wtconv_causal_backward", "wtconv_causal_step")


class SsmTensor(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("batch", ctypes.c_longlong), ("row", ctypes.c_longlong)]


class SelectiveShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "C", "N", "G", "layout", "dtype", "softplus")]


class SelectiveInputs(ctypes.Structure):
    _fields_ = [(n, SsmTensor) for n in ("x", "dt", "Bm", "Cm", "z")] + \
               [(n, ctypes.c_void_p) for n in ("A", "D", "dt_bias", "h0", "lengths")]


class SelectiveGrads(ctypes.Structure):
    _fields_ = [(n, SsmTensor) for n in ("dx", "d_dt", "dB", "dC", "dz")] + \
               [(n, ctypes.c_void_p) for n in ("dA", "dD", "d_dt_bias", "d_h0")]


class CausalShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "C", "K", "layout", "dtype", "silu")]


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
        i, vp, sz, ptr = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
        shape, inputs, tensor, causal = ptr(SelectiveShape), ptr(SelectiveInputs), ptr(SsmTensor), ptr(CausalShape)
        for name, result, arguments in (
                ("wtconv_selective_states_size", sz, [shape]),
                ("wtconv_selective_workspace_size", sz, [i, shape]),
                ("wtconv_selective_forward", i, [shape, inputs, tensor, vp, vp, vp, sz, vp]),
                ("wtconv_selective_backward", i, [shape, inputs, vp, tensor, vp, ptr(SelectiveGrads), vp, sz, vp]),
                ("wtconv_selective_step", i, [shape, inputs, vp, i, vp, tensor, vp]),
                ("wtconv_causal_workspace_size", sz, [causal]),
                ("wtconv_causal_forward", i, [causal, tensor, vp, vp, vp, vp, tensor, vp, vp]),
                ("wtconv_causal_backward", i, [causal, tensor] + [vp] * 4 + [tensor, vp, tensor] + [vp] * 4 + [sz, vp]),
                ("wtconv_causal_step", i, [causal, tensor, vp, vp, vp, i, vp, tensor, vp])):
            getattr(lib, name).restype = result
            getattr(lib, name).argtypes = arguments
        _lib = lib
    return _lib


def wtconv_selective_forward(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None, layout="planes",
                             softplus=True, keep_states=False, y=None, workspace=None, stream=None):
    """(y, h_last, states) of h_t = exp(d_t A) h_{t-1} + d_t x_t B_t, y_t = (C_t . h_t + D x_t) silu(z_t), with
    d = softplus(dt + dt_bias), or dt + dt_bias without ``softplus``.

    A (C, N), D and dt_bias (C,) and h0 (B, C, N) fp32; lengths (B,) int32 ends each sequence.  ``states`` is what
    the backward needs (None unless ``keep_states``); h_last (B, C, N) fp32 is the state after each sequence's
    last position."""
    return (_ext or _load_ext()).selective_forward(x, dt, A, B, C, D, z, dt_bias, h0, lengths, layout, softplus, keep_states, y,
                                                   workspace, stream)


def wtconv_selective_backward(x, dt, A, B, C, states, dy, D=None, z=None, dt_bias=None, dh_last=None, lengths=None,
                              layout="planes", softplus=True, dx=None, d_dt=None, dB=None, dC=None, dz=None, workspace=None,
                              stream=None):
    """(dx, d_dt, dA, dB, dC, dD, dz, d_dt_bias, d_h0) from the forward's inputs and its ``states``; None for what
    belongs to an input that is absent."""
    return (_ext or _load_ext()).selective_backward(x, dt, A, B, C, states, dy, D, z, dt_bias, dh_last, lengths, layout, softplus,
                                                    dx, d_dt, dB, dC, dz, workspace, stream)


def wtconv_selective_step(x, dt, A, B, C, pool, D=None, z=None, dt_bias=None, slots=None, softplus=True, y=None, stream=None):
    """One position of B sequences: x, dt and z (B, C), B and C (B, G, N); updates rows of ``pool`` (n_states, C, N)
    fp32 in place and returns y (B, C).  Sequence b owns slots[b] (int32; b without slots); a slot outside the
    pool marks an idle sequence, whose y is 0."""
    return (_ext or _load_ext()).selective_step(x, dt, A, B, C, pool, D, z, dt_bias, slots, softplus, y, stream)


def wtconv_causal_forward(x, weight, bias=None, state=None, lengths=None, layout="planes", silu=True, y=None, stream=None):
    """(y, state_last) of y_t = silu(bias + sum_k weight_k x_{t-K+1+k}), without ``silu`` the sum itself.

    weight (C, K) with K from 2 to 4 and bias (C,) fp32; state (B, C, K-1) of x's dtype holds the inputs before the
    first position, the oldest first (None: zeros), state_last those before the position after the last one."""
    return (_ext or _load_ext()).causal_forward(x, weight, bias, state, lengths, layout, silu, y, stream)


def wtconv_causal_backward(x, weight, dy, bias=None, state=None, d_last=None, lengths=None, layout="planes", silu=True, dx=None,
                           workspace=None, stream=None):
    """(dx, d_weight, d_bias, d_state) from the forward's inputs; None for the gradient of an absent input.
    d_last (B, C, K-1): the gradient of state_last."""
    return (_ext or _load_ext()).causal_backward(x, weight, dy, bias, state, d_last, lengths, layout, silu, dx, workspace, stream)


def wtconv_causal_step(x, weight, pool, bias=None, slots=None, silu=True, y=None, stream=None):
    """One position of B sequences: x (B, C); updates rows of ``pool`` (n_states, C, K-1) of x's dtype in place and
    returns y (B, C).  Slots as in wtconv_selective_step."""
    return (_ext or _load_ext()).causal_step(x, weight, pool, bias, slots, silu, y, stream)


def _rows(t):
    """A gradient as autograd hands it over, with its innermost axis contiguous."""
    return None if t is None else t.contiguous()


class _Refused(torch.autograd.Function):
    """An operator's gradients as an operation of its own, so that a second derivative meets its refusal."""

    @staticmethod
    def forward(ctx, what, run, *inputs):
        ctx.what = what
        ctx.set_materialize_grads(False)
        return run()

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"the {ctx.what} has no second derivative")


def _gradients(what, run, *inputs):
    """run(), whose results depend on ``inputs``; under ``create_graph`` such that their derivative is refused."""
    return _Refused.apply(what, run, *inputs) if torch.is_grad_enabled() else run()


class WTConvSelectiveFunction(torch.autograd.Function):
    """Autograd wrapper: (y, h_last) through wtconv_selective_forward, gradients through wtconv_selective_backward.
    A derivative of those gradients (``create_graph=True``) is refused.  Without ``keep`` no backward can follow."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, h0, lengths, layout, softplus, keep=True):
        y, h_last, states = wtconv_selective_forward(x, dt, A, B, C, D, z, dt_bias, h0, lengths, layout, softplus,
                                                     keep_states=keep and any(ctx.needs_input_grad))
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, lengths, states)
        ctx.how = layout, softplus
        ctx.h0 = h0  # for its place in the graph only: the backward does not read its values, which may change
        ctx.set_materialize_grads(False)
        return y, h_last

    @staticmethod
    def backward(ctx, dy, dh_last):
        x, dt, A, B, C, D, z, dt_bias, lengths, states = ctx.saved_tensors
        layout, softplus = ctx.how
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _rows(dy)

        def run():
            return wtconv_selective_backward(x, dt, A, B, C, states, dy, D, z, dt_bias, _rows(dh_last), lengths, layout, softplus)

        dx, d_dt, dA, dB, dC, dD, dz, d_bias, d_h0 = _gradients("selective scan", run, x, dt, A, B, C, D, z, dt_bias, ctx.h0, dy, dh_last)
        return dx, d_dt, dA, dB, dC, dD, dz, d_bias, None if ctx.h0 is None else d_h0, None, None, None, None


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lengths=None, layout="planes", softplus=True):
    """Differentiable selective scan: (y, h_last); arguments as wtconv_selective_forward's.  First derivatives only."""
    keep = _recorded(x, dt, A, B, C, D, z, dt_bias, h0)
    return WTConvSelectiveFunction.apply(x, dt, A, B, C, D, z, dt_bias, h0, lengths, layout, softplus, keep)


class WTConvCausalFunction(torch.autograd.Function):
    """Autograd wrapper: (y, state_last) through wtconv_causal_forward, gradients through wtconv_causal_backward.
    A derivative of those gradients (``create_graph=True``) is refused."""

    @staticmethod
    def forward(ctx, x, weight, bias, state, lengths, layout, silu):
        y, last = wtconv_causal_forward(x, weight, bias, state, lengths, layout, silu)
        ctx.save_for_backward(x, weight, bias, state, lengths)
        ctx.how = layout, silu
        ctx.set_materialize_grads(False)
        return y, last

    @staticmethod
    def backward(ctx, dy, d_last):
        x, weight, bias, state, lengths = ctx.saved_tensors
        layout, silu = ctx.how
        dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if dy is None else _rows(dy)

        def run():
            return wtconv_causal_backward(x, weight, dy, bias, state, _rows(d_last), lengths, layout, silu)

        return *_gradients("causal convolution", run, x, weight, bias, state, dy, d_last), None, None, None


def causal_conv(x, weight, bias=None, state=None, lengths=None, layout="planes", silu=True):
    """Differentiable causal convolution: (y, state_last); arguments as wtconv_causal_forward's.  First derivatives only."""
    return WTConvCausalFunction.apply(x, weight, bias, state, lengths, layout, silu)
