"""AdamW in fp64 and the 8-bit state format in NumPy; shares nothing with the CUDA path."""
from __future__ import annotations

import numpy as np

BLOCK = 256
TOP = {"m": 127.0, "v": 255.0}
POWER = {"m": 2, "v": 4}


def step64(p, g, m, v, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, clip=1.0):
    """p', m', v' in fp64."""
    g = np.asarray(g, np.float64) * clip
    m = beta1 * np.asarray(m, np.float64) + (1 - beta1) * g
    v = beta2 * np.asarray(v, np.float64) + (1 - beta2) * g * g
    p = np.asarray(p, np.float64) * (1 - lr * weight_decay) - lr / (1 - beta1 ** step) * m / (
        np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p, m, v


def averages32(g, m, v, beta1=0.9, beta2=0.999):
    """m', v' in fp32, every product and sum rounded by itself."""
    f = np.float32
    g, m, v = (np.asarray(a, f) for a in (g, m, v))
    return f(beta1) * m + f(1 - beta1) * g, f(beta2) * v + f(1 - beta2) * (g * g)


def threshold(n, step):
    i = np.arange(n, dtype=np.uint64)
    u = (i * np.uint64(3242174889) + np.uint64(step) * np.uint64(2447445414)) & np.uint64(0xFFFFFFFF)
    return (u >> np.uint64(8)).astype(np.float32) * np.float32(2.0 ** -24)


def blocks(x):
    n = -(-len(x) // BLOCK) * BLOCK
    return np.concatenate([x, np.zeros(n - len(x), x.dtype)]).reshape(-1, BLOCK)


def held(x, kind, step):
    """Codes and block maxima of the fp32 values x of one tensor, in fp32 arithmetic."""
    f = np.float32
    x = np.asarray(x, f)
    size = blocks(np.abs(x))
    most = size.max(1)
    most = np.where(most < f(2.0 ** -90), f(0), most).astype(f)
    with np.errstate(divide="ignore"):
        inverse = np.where(most > 0, (f(1) / most) * f(TOP[kind] ** POWER[kind]), f(0)).astype(f)
    y = (size * inverse[:, None]).reshape(-1)[:len(x)]

    def level(c):
        return c * c if kind == "m" else (c * c) * (c * c)

    levels = level(np.arange(0, int(TOP[kind]) + 1, dtype=f))
    low = np.clip(np.searchsorted(levels, y, side="right") - 1, 0, int(TOP[kind]) - 1)
    up = (y - levels[low]) > threshold(len(x), step) * (levels[low + 1] - levels[low])
    code = low + up
    if kind == "v":
        return np.where(y > 0, np.maximum(code, 1), code).astype(np.uint8), most
    return (code * np.sign(x)).astype(np.int8), most


def values(code, most, kind):
    """What the codes stand for, in fp64 from the format's formula."""
    c = code.astype(np.float64)
    size = (np.abs(c) / TOP[kind]) ** POWER[kind] * np.repeat(most.astype(np.float64), BLOCK)[:len(c)]
    return size * np.sign(c)
