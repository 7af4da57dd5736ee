"""CPU float64 oracle of the training operators around the attention (test infrastructure).

``qk_norm_rope`` and its backward, the compact-bias attention with masks (a bias of -inf removes its
keys; a row without keys gives zeros and a log-sum-exp of -inf) and its backward from a given
``out`` and ``lse``, and the backward of the projection.  Pinned in ``tests/test_oracle_train.py`` by
central finite differences, closed forms and planted mistakes.
"""
from __future__ import annotations

import numpy as np

from .relpos_oracle import _f64, dense_bias, rel_index


def rotate(y, cos, sin, interleaved: bool, sign: float = 1.0) -> np.ndarray:
    """``y [..., d]`` with its pairs turned by the angles (``cos``, ``sin`` broadcast to ``[..., R / 2]``)."""
    y = _f64(y)
    half = cos.shape[-1]
    z = y.copy()
    ia = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    ib = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = y[..., ia], y[..., ib]
    z[..., ia] = a * cos - sign * b * sin
    z[..., ib] = b * cos + sign * a * sin
    return z


def _angles(cos, sin, positions, B: int, N: int):
    p = np.broadcast_to(np.arange(N), (B, N)) if positions is None else np.asarray(positions)
    return _f64(cos)[p][:, :, None], _f64(sin)[p][:, :, None]


def qk_norm_rope(x, weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                 interleaved: bool = False) -> np.ndarray:
    """One tensor ``x [B, N, heads, d]`` normed and rotated, as ``[B * heads, N, d]``."""
    x = _f64(x)
    B, N, h, d = x.shape
    y = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * _f64(weight)
    if cos is not None:
        y = rotate(y, *_angles(cos, sin, positions, B, N), interleaved)
    return y.transpose(0, 2, 1, 3).reshape(B * h, N, d)


def qk_norm_rope_backward(x, dz, weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                          interleaved: bool = False):
    """Gradients of ``sum(dz * qk_norm_rope(x))``: ``(dx [B, N, heads, d], dweight [d] or None)``."""
    x = _f64(x)
    B, N, h, d = x.shape
    g = _f64(dz).reshape(B, h, N, d).transpose(0, 2, 1, 3)
    if cos is not None:
        g = rotate(g, *_angles(cos, sin, positions, B, N), interleaved, -1.0)
    if weight is None:
        return g.copy(), None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1, 2))
    g = g * _f64(weight)
    return r * (g - x * r * r * (g * x).mean(-1, keepdims=True)), dw


def _logits(q, k, rel_h, rel_w, H, W, scale):
    with np.errstate(invalid="ignore"):
        return scale * (q @ k.T) + dense_bias(rel_h, rel_w, H, W)


def masked_attention(q, k, v, rel_h, rel_w, H: int, W: int, scale: float):
    """``(out [BH, N, d], lse [BH, N] base 2)`` with -inf biases masking."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    out, lse = np.zeros(q.shape), np.empty(q.shape[:2])
    for b in range(q.shape[0]):
        z = _logits(q[b], k[b], _f64(rel_h[b]), _f64(rel_w[b]), H, W, scale)
        top = z.max(-1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        p = np.exp(z - top)
        tot = p.sum(-1, keepdims=True)
        out[b] = p @ v[b] / np.where(tot > 0, tot, 1.0)
        with np.errstate(divide="ignore"):
            lse[b] = (top[:, 0] + np.log(tot[:, 0])) / np.log(2.0)
    return out, lse


def attention_backward_from(q, k, v, rel_h, rel_w, out, lse, dout, H: int, W: int, scale: float):
    """``(dq, dk, dv, drel_h, drel_w)`` with P from the given base-2 ``lse`` and D from the given ``out``.  On an axis
    of length one the bias's gradient is zero whatever rounding ``out`` and ``lse`` have seen."""
    q, k, v, out, lse, dout = (_f64(t) for t in (q, k, v, out, lse, dout))
    BH, N, _ = q.shape
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dh, dw = np.zeros((BH, N, H)), np.zeros((BH, N, W))
    for b in range(BH):
        z = _logits(q[b], k[b], _f64(rel_h[b]), _f64(rel_w[b]), H, W, scale)
        some = np.isfinite(lse[b])
        p = np.exp(z - np.where(some, lse[b], 0.0)[:, None] * np.log(2.0)) * some[:, None]
        dv[b] = p.T @ dout[b]
        dz = p * (dout[b] @ v[b].T - (dout[b] * out[b]).sum(-1, keepdims=True))
        dq[b] = scale * (dz @ k[b])
        dk[b] = scale * (dz.T @ q[b])
        grid = dz.reshape(N, H, W)
        dh[b], dw[b] = grid.sum(2) * (H > 1), grid.sum(1) * (W > 1)
    return dq, dk, dv, dh, dw


def project_backward(q, rel_pos_h, rel_pos_w, drel_h, drel_w, H: int, W: int):
    """Gradients of ``sum(drel_h * rel_h + drel_w * rel_w)``: ``(dq, drel_pos_h, drel_pos_w)``."""
    q, th, tw = _f64(q), _f64(rel_pos_h), _f64(rel_pos_w)
    BH, N, d = q.shape
    dq, dth, dtw = np.zeros((BH, H, W, d)), np.zeros_like(th), np.zeros_like(tw)
    qg = q.reshape(BH, H, W, d)
    gh, gw = _f64(drel_h).reshape(BH, H, W, H), _f64(drel_w).reshape(BH, H, W, W)
    ih, iw = rel_index(H), rel_index(W)
    for a in range(H):
        dq[:, a] += gh[:, a] @ th[ih[a]]
        np.add.at(dth, ih[a], np.einsum("bwk,bwc->kc", gh[:, a], qg[:, a]))
    for a in range(W):
        dq[:, :, a] += gw[:, :, a] @ tw[iw[a]]
        np.add.at(dtw, iw[a], np.einsum("bhk,bhc->kc", gw[:, :, a], qg[:, :, a]))
    return dq.reshape(BH, N, d), dth, dtw
