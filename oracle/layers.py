"""Plain CPU float64 oracle of the operators ahead of the output head.

TEST INFRASTRUCTURE ONLY (see ``oracle/kl.py``): nothing on the product path imports it.

    rmsnorm       h = x + residual, y = h / sqrt(mean_j h_j^2 + eps) * gamma
    e4m3 rows     scale = max_j |y_j| / 448, q = e4m3(y / scale)
    linear        z = x W^T + bias, y = act(z) + residual
    gradients     by the chain rule, written out per element

Arguments and results are float64 arrays.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")

_erf = np.vectorize(math.erf, otypes=[np.float64])


def rmsnorm(x, residual, gamma, eps):
    """(h, y)."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * gamma


def rmsnorm_grad(dy, h, gamma, eps, dh=None):
    """(dx, dgamma): the vector-Jacobian product of rmsnorm at h, and dh added to dx."""
    rms = np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    xhat = h / rms
    a = dy * gamma
    dx = (a - xhat * (a * xhat).mean(axis=1, keepdims=True)) / rms
    return (dx if dh is None else dx + dh), (dy * xhat).sum(axis=0)


def e4m3_values():
    """Every finite value of the 8-bit format with 4 exponent and 3 mantissa bits (bias 7, largest 448)."""
    v = []
    for e in range(16):
        for m in range(8):
            if e == 15 and m == 7:
                continue                      # NaN
            v.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(sorted(set(v) | {-u for u in v}))


def e4m3_rows(y):
    """(values the rows are held as, scale): value = scale * nearest e4m3 of y / scale, ties to the even mantissa."""
    table = e4m3_values()
    pos = table[table >= 0]                   # index parity = parity of the mantissa's last bit
    scale = np.abs(y).max(axis=1) / E4M3_MAX
    q = np.zeros_like(y)
    for n in range(y.shape[0]):
        if scale[n] == 0:
            continue
        t = np.minimum(np.abs(y[n]) / scale[n], E4M3_MAX)
        hi = np.clip(np.searchsorted(pos, t), 1, len(pos) - 1)
        lo = hi - 1
        dl, dh = t - pos[lo], pos[hi] - t
        take = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
        q[n] = np.sign(y[n]) * pos[take]
    return q, scale


def act(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    assert kind == "silu"
    return z / (1.0 + np.exp(-z))


def act_grad(z, kind):
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)     # 0 at 0
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    assert kind == "silu"
    s = 1.0 / (1.0 + np.exp(-z))
    return s + z * s * (1.0 - s)


def linear(x, W, bias=None, residual=None, kind="none"):
    """(y, z)."""
    z = x @ W.T
    if bias is not None:
        z = z + bias
    y = act(z, kind)
    return (y if residual is None else y + residual), z


def linear_grad(dy, pre, x, W, kind="none"):
    """(dx, dW, dbias, dz) at the pre-activation `pre`."""
    dz = dy * act_grad(pre, kind) if kind != "none" else dy
    return dz @ W, dz.T @ x, dz.sum(axis=0), dz
