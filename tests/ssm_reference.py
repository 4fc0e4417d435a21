"""The selective scan and the causal convolution in fp64, position by position, with NumPy, and bounds of what fp32
may make of them; shares nothing with the CUDA path.

Arrays are time first: x, dt, z, dy (T, B, C); Bm, Cm (T, B, G, N); A (C, N); D, dt_bias (C,); h0, dh_last (B, C, N);
lengths (B,).  Every result comes with a bound on its error in fp32, carried along the recurrences: with
u = 2^-24, half a unit of a value's last place relative to it,

  exp2, reciprocal   off by 2 units of the last place at most, 4u;
  d = softplus(v)    v is rounded (u |v|), and so are v log2 e and log2 e itself (2u |v|), which reach e = exp(-|v|);
                     exp2 4u, a quotient 5u, the series and the sum 5u: (3 |v| + 14) u relative to d, and to sigmoid(v)
  silu(z)            z log2 e twice u |z|, exp2 4u, the sum, reciprocal and product 6u: (2 |z| + 10) u
  a = exp2(d A')     the argument is off by d's error, that of A' = A log2 e (u) and the product's (u); exp2 4u
  h = a h + b        the product is not rounded on its own: u of the result
  sums over N states or lanes   at most 8u of the sum of absolute values (7 additions in a row, products fused)
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HALF_UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # finfo.eps / 2


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def silu_slope(v):
    p = sigmoid(v)
    return p * (1 + v * (1 - p))


def ends_of(lengths, T, B):
    return np.full(B, T) if lengths is None else np.clip(lengths, 0, T)


def selective(d):
    """All results of a forward and a backward as {name: (value, bound)}; d: dict of the arrays above, those that
    are absent None, and softplus."""
    x, raw, A, Bm, Cm, D, z, bias, h0, dy, dh = (d[k] for k in ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0", "dy", "dh_last"))
    T, B, C = x.shape
    N, G = A.shape[1], Bm.shape[2]
    ends = ends_of(d["lengths"], T, B)
    live = (np.arange(T)[:, None] < ends)[:, :, None]
    zero = lambda v: np.where(live if v.ndim == 3 else live[..., None], v, 0.0)  # noqa: E731
    x, raw, Bm, Cm, dy = zero(x), zero(raw), zero(Bm), zero(Cm), zero(dy)
    group = np.arange(C) // (C // G)
    Bc, Cc = Bm[:, :, group], Cm[:, :, group]                 # (T, B, C, N)
    v = raw if bias is None else raw + bias
    if d["softplus"]:
        step, slope = np.logaddexp(0, v), sigmoid(v)
        rd = (3 * np.abs(v) + 14) * U
    else:
        step, slope, rd = v, np.ones_like(v), np.full_like(v, 0 if bias is None else np.nan)
        if bias is not None:
            rd = U * np.ones_like(v)
    step, rd = zero(step), zero(rd)
    arg = step[..., None] * A
    a = np.exp(arg)
    ra = np.abs(arg) * (rd[..., None] + 3 * U) + 6 * U
    ra = zero(ra)
    drive = (step * x)[..., None] * Bc
    h, H, E = np.zeros((T + 1, B, C, N)), np.zeros((T + 1, B, C, N)), np.zeros((T + 1, B, C, N))
    if h0 is not None:
        h[0], H[0] = h0, np.abs(h0)
    for t in range(T):
        h[t + 1] = np.where(live[t][..., None], a[t] * h[t] + drive[t], h[t])
        H[t + 1] = np.where(live[t][..., None], a[t] * H[t] + np.abs(drive[t]), H[t])
        e = a[t] * E[t] + ra[t] * a[t] * H[t] + (rd[t][..., None] + 4 * U) * np.abs(drive[t]) + U * H[t + 1]
        E[t + 1] = np.where(live[t][..., None], e, E[t])
    out = (Cc * h[1:]).sum(-1)
    out_abs, out_err = (np.abs(Cc) * H[1:]).sum(-1), (np.abs(Cc) * (E[1:] + 8 * U * H[1:])).sum(-1)
    if D is not None:
        out, out_abs = out + D * x, out_abs + np.abs(D * x)
        out_err = out_err + 2 * U * out_abs
    gate, gate_err = np.ones_like(x), np.zeros_like(x)
    if z is not None:
        z = zero(z)
        gate, gate_err = z * sigmoid(z), (2 * np.abs(z) + 10) * U
    res = {"y": (zero(out * gate), np.abs(gate) * (out_err + out_abs * (gate_err + U))),
           "h_last": (h[T], E[T])}
    r, rr = dy * gate, gate_err + U
    g, Gm, EG = np.zeros_like(a), np.zeros_like(a), np.zeros_like(a)
    flow = np.zeros((B, C, N)) if dh is None else dh.astype(np.float64)
    Flow, EF = np.abs(flow), np.zeros_like(flow)
    for t in reversed(range(T)):
        on = live[t][..., None]
        into = r[t][..., None] * Cc[t]
        g[t] = np.where(on, into + flow, 0.0)
        Gm[t] = np.where(on, np.abs(into) + Flow, 0.0)
        EG[t] = np.where(on, np.abs(into) * (rr[t][..., None] + 2 * U) + EF + U * Gm[t], 0.0)
        flow = np.where(on, a[t] * g[t], flow)
        EF = np.where(on, a[t] * (EG[t] + Gm[t] * (ra[t] + U)), EF)
        Flow = np.where(on, a[t] * Gm[t], Flow)
    per_group = lambda q: q.reshape(T, B, G, C // G, N).sum(3)  # noqa: E731
    many = (C // G + 8) * U                                       # a sum over the channels of a group
    res["dC"] = (per_group(zero(r[..., None] * h[1:])), per_group(zero(np.abs(r)[..., None] * (E[1:] + H[1:] * (rr[..., None] + many)))))
    dx_abs = np.abs(step * x)[..., None]
    res["dB"] = (per_group((step * x)[..., None] * g), per_group(dx_abs * (EG + Gm * (rd[..., None] + many))))
    # In bf16 the products that dB and dC sum are cut to 11 bits, and the sum gets a factor 1 + f, f = 3 x 2^-13.  With m 2^e,
    # 1 <= m < 2, cutting loses l 2^e with 0 <= l < 2^-10; (m - l) (1 + f) / m - 1 = f - (1 + f) l / m lies between f -
    # (1 + f) 2^-10 = -6.107e-4 and f = 3.663e-4.
    res["cut"] = {"dC": 6.11e-4 * per_group(zero(np.abs(r[..., None] * h[1:]))), "dB": 6.11e-4 * per_group(dx_abs * np.abs(g))}
    into, into_abs, into_err = (g * Bc).sum(-1), (Gm * np.abs(Bc)).sum(-1), (np.abs(Bc) * (EG + 8 * U * Gm)).sum(-1)
    dx, dx_err = step * into, step * (into_err + into_abs * (rd + 2 * U))
    if D is not None:
        dx = dx + D * r
        dx_err = dx_err + np.abs(D * r) * (rr + 2 * U) + U * np.abs(dx)
    res["dx"] = (zero(dx), dx_err)
    k, K = g * a * h[:-1], Gm * a * H[:-1]
    EK = a * (EG * H[:-1] + Gm * E[:-1]) + K * (ra + 3 * U)
    dd = (k * A).sum(-1) + x * into
    dd_abs = (K * np.abs(A)).sum(-1) + np.abs(x) * into_abs
    dd_err = (np.abs(A) * (EK + 10 * U * K)).sum(-1) + np.abs(x) * into_err + 3 * U * dd_abs
    res["d_dt"] = (zero(dd * slope), zero(slope * (dd_err + dd_abs * (rd + 2 * U))))
    terms = (T / 2 + 40 + B) * U                                  # sums over positions: at most T / 2 in a row
    res["dA"] = ((k * step[..., None]).sum((0, 1)), (step[..., None] * (EK + K * (rd[..., None] + terms))).sum((0, 1)))
    res["d_dt_bias"] = (res["d_dt"][0].sum((0, 1)), (res["d_dt"][1] + terms * np.abs(res["d_dt"][0])).sum((0, 1)))
    res["dD"] = ((r * x).sum((0, 1)), (np.abs(r * x) * (rr + terms)).sum((0, 1)))
    res["dz"] = (zero(dy * out * (1 if z is None else silu_slope(z))),
                 np.abs(dy) * (out_err * 1.1 + out_abs * ((0 if z is None else 2 * np.abs(z) + 14) * U) * 1.1))
    res["d_h0"] = (flow, EF)
    return res


def causal(d):
    """As selective(); d: x, dy (T, B, C), w (C, K), bias, state (B, C, K-1), d_last, lengths, silu."""
    x, dy, w, state = d["x"], d["dy"], d["w"], d["state"]
    T, B, C = x.shape
    K = w.shape[1]
    ends = ends_of(d["lengths"], T, B)
    live = (np.arange(T)[:, None] < ends)[:, :, None]
    x, dy = np.where(live, x, 0.0), np.where(live, dy, 0.0)
    seen = np.concatenate([np.zeros((K - 1, B, C)) if state is None else state.transpose(2, 0, 1), x])
    bias = np.zeros(C) if d["bias"] is None else d["bias"]
    pre, pre_abs = np.broadcast_to(bias, x.shape).copy(), np.broadcast_to(np.abs(bias), x.shape).copy()
    for k in range(K):
        pre += w[:, k] * seen[k:k + T]
        pre_abs += np.abs(w[:, k] * seen[k:k + T])
    err = K * U * pre_abs                                         # K fused products
    f, slope, fe, se = pre, np.ones_like(pre), err, np.zeros_like(pre)
    if d["silu"]:
        f, slope = pre * sigmoid(pre), silu_slope(pre)
        fe = 1.1 * err + np.abs(f) * (2 * np.abs(pre) + 10) * U   # |silu'| < 1.1, |silu''| <= 1/2
        se = 0.5 * err + (2 * np.abs(pre) + 14) * U * 1.1
    res = {"y": (np.where(live, f, 0.0), fe)}
    g, ge = dy * slope, np.abs(dy) * (se + 2 * U)
    d_seen, de = np.zeros_like(seen), np.zeros_like(seen)
    dw, dwe = np.zeros_like(w), np.zeros_like(w)
    terms = (T + B + 40) * U
    for k in range(K):
        d_seen[k:k + T] += w[:, k] * g
        de[k:k + T] += np.abs(w[:, k]) * (ge + (K + 1) * U * np.abs(g))
        dw[:, k] = (g * seen[k:k + T]).sum((0, 1))
        dwe[:, k] = (np.abs(seen[k:k + T]) * (ge + terms * np.abs(g))).sum((0, 1))
    last = np.zeros((B, C, K - 1))
    for b in range(B):
        last[b] = seen[ends[b]:ends[b] + K - 1, b].T
        if d["d_last"] is not None:
            d_seen[ends[b]:ends[b] + K - 1, b] += d["d_last"][b].T
    de += U * np.abs(d_seen)
    dx = np.where(live, d_seen[K - 1:], 0.0)
    res.update(last=(last, np.zeros_like(last)), dx=(dx, de[K - 1:]), dw=(dw, dwe),
               d_bias=(g.sum((0, 1)), (ge + terms * np.abs(g)).sum((0, 1))),
               d_state=(d_seen[:K - 1].transpose(1, 2, 0), de[:K - 1].transpose(1, 2, 0)))
    return res


def assert_within(name, got, value, bound, dtype=torch.float32):
    """|got - value| <= bound, and half a unit of dtype for the rounding when it is stored."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == value.shape, f"{name}: shape {got.shape}, expected {value.shape}"
    assert np.isfinite(got).all(), f"{name}: non-finite values"
    # a 16-bit value below the least normal one is off by half its last place at most; 1.01: products of errors
    least = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -126}[dtype]
    allowed = 1.01 * (bound + HALF_UNIT[dtype] * (np.abs(value) + bound)) + least
    worst = np.max(np.abs(got - value) - allowed) if got.size else 0.0
    assert worst <= 0, f"{name}: off by {np.max(np.abs(got - value)):.3e}, {worst:.3e} over the bound"
