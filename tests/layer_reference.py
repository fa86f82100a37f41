"""Plain 64-bit forms of the norm, the rotary positions and the gated feed-forward with their gradients, in
numpy. They share nothing with the library but the formulas of include/fp4.h."""
import math

import numpy as np


def rmsnorm(s, w, eps):
    return s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * w


def rmsnorm_grad(dy, s, w, eps, dsum=0.0):
    r = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    n, a = s * r, dy * w
    return dsum + r * (a - n * (a * n).mean(1, keepdims=True)), (dy * n).sum(0)


def rope(x, pos, inv_freq, interleaved, scale=1.0, backward=False):
    """x [tokens, heads, dim]."""
    y = x.copy()
    n = len(inv_freq)
    for t in range(x.shape[0]):
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            angle = float(pos[t]) * float(inv_freq[i])
            c, s = math.cos(angle), math.sin(angle) * (-1.0 if backward else 1.0)
            y[t, :, a] = scale * (x[t, :, a] * c - x[t, :, b] * s)
            y[t, :, b] = scale * (x[t, :, b] * c + x[t, :, a] * s)
    return y


_erf = np.vectorize(math.erf)


def act(g, kind):
    if kind == 0:
        with np.errstate(over="ignore"):
            return g / (1.0 + np.exp(-g))
    if kind == 1:
        return 0.5 * g * (1.0 + _erf(g / math.sqrt(2.0)))
    return 0.5 * g * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))


def act_grad(g, kind):
    if kind == 0:
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-g))
        return p + g * p * (1.0 - p)
    if kind == 1:
        return 0.5 * (1.0 + _erf(g / math.sqrt(2.0))) + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    t = np.tanh(z)
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * g * g)


def gated_grad(dh, g, u, kind):
    return np.concatenate([dh * u * act_grad(g, kind), dh * act(g, kind)], 1)
