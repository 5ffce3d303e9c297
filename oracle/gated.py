"""Plain 64-bit definitions of the gated feed-forward block's operators (numpy): the gated linear
layer, the norms before and after a block with its gate and residual scale, low-rank adapters.
Test infrastructure only; it shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

ACTS = ("silu", "gelu", "gelu_tanh", "sigmoid", "relu", "relu2", "identity")
_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1 / (1 + e), e / (1 + e))


def activation(g, act: str):
    """(f(g), f'(g))."""
    if act == "silu":
        p = sigmoid(g)
        return g * p, p + g * p * (1 - p)
    if act == "gelu":
        phi = 0.5 * _erfc(-g / math.sqrt(2))
        return g * phi, phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        p = sigmoid(2 * c * (g + 0.044715 * g ** 3))
        return g * p, p + g * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * g * g)
    if act == "sigmoid":
        p = sigmoid(g)
        return p, p * sigmoid(-g)
    if act == "relu":
        return np.maximum(g, 0), (g > 0).astype(np.float64)
    if act == "relu2":
        r = np.maximum(g, 0)
        return r * r, 2 * r
    return g, np.ones_like(g)


def gated_linear(x, w_gate, w_up, act: str):
    """(h, g, u)."""
    g, u = x @ w_gate.T, x @ w_up.T
    return activation(g, act)[0] * u, g, u


def gated_linear_backward(dh, g, u, x, w_gate, w_up, act: str):
    """(dx, dw_gate, dw_up)."""
    f, slope = activation(g, act)
    dg, du = dh * u * slope, dh * f
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x


def rms_inverse(v, eps: float):
    return 1.0 / np.sqrt((v * v).mean(1) + eps)


def block_norm(x, residual, post, gate, pre, eps, a, b, stored=lambda z: z):
    """(z, y, post_rstd, pre_rstd); `stored` rounds z as the second norm reads it."""
    r1 = None if x is None else rms_inverse(x, eps)
    z = residual if x is None else a * residual + b * gate * x * r1[:, None] * post
    v = stored(z)
    r2 = rms_inverse(v, eps)
    return z, v * r2[:, None] * pre, r1, r2


def block_norm_backward(dy, dz_add, x, z, post, gate, pre, r1, r2, a, b):
    """(dresidual, dx, dgate per token and channel, dpost, dpre)."""
    dz, dpre = dz_add, None
    if dy is not None:
        zh, c = z * r2[:, None], dy * pre
        dz = dz + r2[:, None] * (c - zh * (c * zh).mean(1, keepdims=True))
        dpre = (dy * zh).sum(0)
    if x is None:
        return dz, None, None, None, dpre
    xh = x * r1[:, None]
    e = b * gate * dz
    q = e * post
    dx = r1[:, None] * (q - xh * (q * xh).mean(1, keepdims=True))
    return a * dz, dx, b * dz * xh * post, (e * xh).sum(0), dpre


def lora_add(x, a, b, scale, index, base, ranks=None):
    """y, and the sum of the magnitudes its low-rank part is made of."""
    y = base.copy()
    size = np.zeros_like(base)
    for t, i in enumerate(index):
        if not 0 <= i < len(a):
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        v = a[i, :r] @ x[t]
        y[t] += scale[i] * (b[i, :, :r] @ v)
        size[t] = abs(scale[i]) * (np.abs(b[i, :, :r]) @ (np.abs(a[i, :r]) @ np.abs(x[t])))
    return y, size
