"""The gated scan in fp64, position by position, with NumPy; shares nothing with the CUDA path.

Arrays are time first: x, gate, dy (T, B, C); gate_bias (C,); h0, dh_last (B, C); lengths (B,)."""
from __future__ import annotations

import numpy as np
import torch


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def forward(x, gate, gate_bias, h0=None, lengths=None):
    """y, h_last and the state before every position (T, B, C)."""
    T, B, C = x.shape
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    h = np.zeros((B, C)) if h0 is None else np.array(h0, np.float64)
    y, before = np.zeros((T, B, C)), np.zeros((T, B, C))
    for t in range(T):
        before[t] = h
        live = (t < n)[:, None]
        a = sigmoid(np.where(live, gate[t], 0.0) + gate_bias)
        h = np.where(live, a * h + (1 - a) * np.where(live, x[t], 0.0), h)
        y[t] = np.where(live, h, 0.0)
    return y, h, before


def backward(x, gate, gate_bias, dy, h0=None, dh_last=None, lengths=None):
    """dict dx, d_gate, d_gate_bias, d_h0, and the sum of |d_gate| that d_gate_bias cancels in."""
    T, B, C = x.shape
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    _, _, before = forward(x, gate, gate_bias, h0, lengths)
    flow = np.zeros((B, C)) if dh_last is None else np.array(dh_last, np.float64)
    dx, dg = np.zeros((T, B, C)), np.zeros((T, B, C))
    for t in reversed(range(T)):
        live = (t < n)[:, None]
        a = sigmoid(np.where(live, gate[t], 0.0) + gate_bias)
        dh = np.where(live, dy[t], 0.0) + flow
        dx[t] = np.where(live, (1 - a) * dh, 0.0)
        dg[t] = np.where(live, dh * (before[t] - np.where(live, x[t], 0.0)) * a * (1 - a), 0.0)
        flow = np.where(live, a * dh, flow)
    return {"dx": dx, "d_gate": dg, "d_gate_bias": dg.sum((0, 1)), "d_h0": flow, "abs": np.abs(dg).sum((0, 1))}


def time_first(t: torch.Tensor, layout: str) -> np.ndarray:
    """A GPU activation in either layout as a (T, B, C) fp64 array."""
    a = t.detach().double().cpu().numpy()
    if a.ndim == 4:
        a = a.reshape(*a.shape[:2], -1)
    return a.transpose(1, 0, 2) if layout == "tokens" else a.transpose(2, 0, 1)


# Bounds.  An activation is rounded once: half a unit of its type relative to the value (24, 8 and 11
# significant bits).  Beside it, fp32: a gate is off by a few 2^-24, at random, and a state remembers
# up to ~500 of them (gates up to sigmoid(6 + 3)): sqrt(500) * 4 * 2^-24 = 5e-6 of the largest value;
# 1e-5 is allowed.
HALF_UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F32_BOUND = 1e-5


def assert_near(name, got: np.ndarray, want: np.ndarray, dtype=torch.float32, scale=None):
    """|got - want| <= half a unit of dtype |want| + F32_BOUND * scale (the largest |want| by default)."""
    assert got.shape == want.shape, f"{name}: shape {got.shape}, expected {want.shape}"
    assert np.isfinite(got).all(), f"{name}: non-finite values"
    if scale is None:
        scale = np.abs(want).max() if want.size else 0.0
    # a 16-bit value below the least normal one is off by half its last place at most
    bound = HALF_UNIT[dtype] * 1.01 * np.abs(want) + F32_BOUND * scale + (2.0 ** -25 if dtype == torch.float16 else 0)
    worst = np.max(np.abs(got - want) - bound)
    assert worst <= 0, f"{name}: off by {np.max(np.abs(got - want)):.3e}, {worst:.3e} over the bound"
