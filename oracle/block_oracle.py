"""float64 reference of the encoder block's norms, linear layers and activations.

Written from the formulas in NumPy; shares no code with the package.
"""
from __future__ import annotations

import math

import numpy as np



def _erfc(x):
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


def layer_norm(x, weight=None, bias=None, eps=1e-6):
    """(y, mean, rstd) of [..., C]."""
    mean = x.mean(-1)
    xc = x - mean[..., None]
    rstd = 1.0 / np.sqrt((xc * xc).mean(-1) + eps)
    y = xc * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, dres=None):
    """(dx, dweight, dbias) with the statistics as given."""
    h = (x - mean[..., None]) * rstd[..., None]
    g = dy if weight is None else dy * weight
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - h * (g * h).mean(-1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * h).sum(axes), dy.sum(axes)


def activation(u, act):
    if act is None:
        return u
    if act == "relu":
        return np.maximum(u, 0.0)
    if act == "gelu":
        return 0.5 * u * _erfc(-u / math.sqrt(2.0))
    if act == "gelu_tanh":
        return 0.5 * u * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (u + 0.044715 * u ** 3)))
    c = {"quick_gelu": 1.702, "silu": 1.0}[act]
    return u * 0.5 * (1.0 + np.tanh(0.5 * c * u))


def activation_slope(u, act):
    if act is None:
        return np.ones_like(u)
    if act == "relu":
        return (u > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * _erfc(-u / math.sqrt(2.0)) + u * np.exp(-0.5 * u * u) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        b = math.sqrt(2.0 / math.pi)
        t = np.tanh(b * (u + 0.044715 * u ** 3))
        return 0.5 * (1.0 + t) + 0.5 * u * (1.0 - t * t) * b * (1.0 + 3 * 0.044715 * u * u)
    c = {"quick_gelu": 1.702, "silu": 1.0}[act]
    s = 0.5 * (1.0 + np.tanh(0.5 * c * u))
    return s + c * u * s * (1.0 - s)


def linear(x, weight, bias=None, act=None, residual=None):
    """(y, pre) of tokens [M, K]."""
    u = x @ weight.T
    if bias is not None:
        u = u + bias
    y = activation(u, act)
    return (y if residual is None else y + residual), u


def linear_backward(dy, x, weight, input_pre=None, input_act=None):
    """(dx, dweight, dbias) of tokens [M, K], [M, out]."""
    dx = dy @ weight
    if input_pre is not None:
        dx = dx * activation_slope(input_pre, input_act)
    return dx, dy.T @ x, dy.sum(0)
