"""What the block's kernels may be off by, from their arithmetic (float64 arrays throughout)."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import block_oracle as ob

HF = torch.float16


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def rounding(want, dtype):
    """Half a step of the output's type (fp16 subnormals: 2^-25)."""
    return torch.finfo(dtype).eps / 2 * np.abs(want) + (2.0 ** -25 if dtype == HF else 2.0 ** -130)


def product(a, b):
    """Of sums of products of 16-bit values, a b^T: the products are exact; the tensor core adds 16 at a time to its fp32 sum and
    cuts what that leaves, at most 2^-22 of the largest partial sum, which the sum of the sizes bounds; eight more for
    sums of pieces and the epilogue."""
    return (a.shape[1] / 16 + 8) * 2.0 ** -22 * (np.abs(a) @ np.abs(b).T)


def _sigmoid(u, act):
    """(s, its argument's size, the factor of s (1 - s) in the slope)"""
    if act == "gelu_tanh":
        b = 2 * math.sqrt(2 / math.pi)
        v = b * (u + 0.044715 * u ** 3)
        return 0.5 * (1 + np.tanh(0.5 * v)), np.abs(v), np.abs(b * u * (1 + 3 * 0.044715 * u * u))
    c = {"quick_gelu": 1.702, "silu": 1.0}[act]
    return 0.5 * (1 + np.tanh(0.5 * c * u)), np.abs(c * u), np.abs(c * u)


def _ds(s, v):
    """Of a sigmoid: its argument is off by 2^-22 relative (three roundings), the exponential and the reciprocal by
    2^-21 together."""
    return s * (1 - s) * (v * 2.0 ** -21 + 2.0 ** -20) + 2.0 ** -21 * s


def _dtail(u):
    """Of Phi(-|u|): the fit's 2^-20, the polynomial's eight roundings, the reciprocal and the exponential 2^-20 together, and
    the exponential's argument, u^2 / 2 off by 2^-22 relative."""
    return 0.5 * np.vectorize(math.erfc)(np.abs(u) / math.sqrt(2)) * (2.0 ** -18 + u * u * 2.0 ** -22)


def act(u, name):
    """Of an activation in fp32 (2^-22: the roundings of the result's own product and sum)."""
    if name in (None, "relu"):
        return np.zeros_like(u)
    own = 2.0 ** -22 * np.abs(ob.activation(u, name)) + 2.0 ** -120
    if name == "gelu":
        return np.abs(u) * _dtail(u) + own
    s, v, _ = _sigmoid(u, name)
    return np.abs(u) * _ds(s, v) + own


def slope(u, name):
    """Of an activation's derivative in fp32."""
    if name in (None, "relu"):
        return np.zeros_like(u)
    own = 2.0 ** -22 * np.abs(ob.activation_slope(u, name)) + 2.0 ** -23
    if name == "gelu":
        return _dtail(u) + np.abs(u) * np.exp(-0.5 * u * u) * (2.0 ** -20 + u * u * 2.0 ** -22) + own
    s, v, m = _sigmoid(u, name)
    return (1 + m) * _ds(s, v) + m * s * 2.0 ** -24 + own


def near(got, want, tol, what):
    g = f64(got)
    assert g.shape == want.shape, f"{what}: {g.shape}, expected {want.shape}"
    assert np.isfinite(g).all(), f"{what}: not finite"
    over = np.abs(g - want) - tol
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over its tolerance at {np.unravel_index(over.argmax(), over.shape)}"
