"""Pins of the training operators' oracle (no GPU): central finite differences of every gradient, closed
forms, and planted mistakes that the differences catch."""
from __future__ import annotations

import numpy as np
import pytest

import oracle


def fd(loss, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        xp, xm = x.copy(), x.copy()
        xp[i] += h
        xm[i] -= h
        g[i] = (loss(xp) - loss(xm)) / (2 * h)
    return g


def near(a, b):
    return np.abs(a - b).max() <= 1e-6 * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_qk_norm_rope_gradients(inter, norm):
    r = np.random.default_rng(0)
    B, N, h, d, R = 2, 3, 2, 6, 4
    x, w = r.standard_normal((B, N, h, d)), (1 + 0.3 * r.standard_normal(d) if norm else None)
    ang = r.standard_normal((7, R // 2))
    kw = dict(cos=np.cos(ang), sin=np.sin(ang), positions=r.integers(0, 7, (B, N)), eps=0.1, interleaved=inter)
    dz = r.standard_normal((B * h, N, d))
    dx, dw = oracle.qk_norm_rope_backward(x, dz, w, **kw)
    assert near(dx, fd(lambda t: float((dz * oracle.qk_norm_rope(t, w, **kw)).sum()), x))
    if norm:
        assert near(dw, fd(lambda t: float((dz * oracle.qk_norm_rope(x, t, **kw)).sum()), w))
    # planted: the angle's sign, and the norm's mean left out
    bad, _ = oracle.qk_norm_rope_backward(x, dz, w, **{**kw, "sin": -kw["sin"]})
    assert not near(bad, dx)


def test_rotation_closed_forms():
    r = np.random.default_rng(1)
    y, a = r.standard_normal((5, 8)), r.standard_normal((5, 3))
    for inter in (False, True):
        z = oracle.rotate(y, np.cos(a), np.sin(a), inter)
        assert np.allclose(np.linalg.norm(z, axis=-1), np.linalg.norm(y, axis=-1))     # lengths are kept
        assert np.array_equal(z[:, 6:], y[:, 6:])                                       # the rest passes
        assert np.allclose(oracle.rotate(z, np.cos(a), np.sin(a), inter, -1.0), y)
        back = oracle.rotate(oracle.rotate(y, np.cos(a), np.sin(a), inter), np.cos(a), np.sin(a), inter)
        assert np.allclose(back, oracle.rotate(y, np.cos(2 * a), np.sin(2 * a), inter))
    # a quarter turn takes (1, 0) to (0, 1), in both pairings
    e = np.eye(4)[:1]
    assert np.allclose(oracle.rotate(e, np.zeros((1, 2)), np.ones((1, 2)), False), np.eye(4)[2:3])
    assert np.allclose(oracle.rotate(e, np.zeros((1, 2)), np.ones((1, 2)), True), np.eye(4)[1:2])


def test_masked_attention():
    r = np.random.default_rng(2)
    BH, H, W, d = 2, 3, 4, 4
    N = H * W
    q, k, v, do = (r.standard_normal((BH, N, d)) for _ in range(4))
    rh, rw = r.standard_normal((BH, N, H)), r.standard_normal((BH, N, W))
    out, lse = oracle.masked_attention(q, k, v, rh, rw, H, W, 0.5)
    assert np.allclose(out, oracle.attention(q, k, v, rh, rw, H, W, 0.5))
    assert np.allclose(lse, oracle.lse2(q, k, rh, rw, H, W, 0.5))
    want = oracle.attention_backward(q, k, v, rh, rw, H, W, 0.5, do)
    for a, b in zip(oracle.attention_backward_from(q, k, v, rh, rw, out, lse, do, H, W, 0.5), want):
        assert np.allclose(a, b)
    # the last grid row and column masked: the smaller grid's attention; one row without keys
    rh[:, :, 2], rw[:, :, 3] = -np.inf, -np.inf
    rh[0, 5] = -np.inf
    out, lse = oracle.masked_attention(q, k, v, rh, rw, H, W, 0.5)
    keys = [kh * W + kw for kh in range(2) for kw in range(3)]
    z = 0.5 * q[1] @ k[1][keys].T + (rh[1][:, :2, None] + rw[1][:, None, :3]).reshape(N, -1)
    p = np.exp(z) / np.exp(z).sum(-1, keepdims=True)
    assert np.allclose(out[1], p @ v[1][keys])
    assert np.all(out[0, 5] == 0) and lse[0, 5] == -np.inf
    grads = oracle.attention_backward_from(q, k, v, rh, rw, out, lse, do, H, W, 0.5)

    def loss(**x):
        a = dict(q=q, k=k, v=v, rel_h=rh, rel_w=rw)
        a.update(x)
        return float((do * oracle.masked_attention(a["q"], a["k"], a["v"], a["rel_h"], a["rel_w"], H, W, 0.5)[0]).sum())

    for name, x, g in zip(("q", "k", "v"), (q, k, v), grads):
        assert near(g, fd(lambda t, name=name: loss(**{name: t}), x)), name
    assert all(np.isfinite(g).all() for g in grads)
    assert np.all(grads[0][0, 5] == 0) and np.all(grads[3][0, 5] == 0)
    assert np.all(grads[1][:, [n for n in range(N) if n not in keys]] == 0)


def test_project_backward_gradients():
    r = np.random.default_rng(3)
    BH, H, W, d = 2, 2, 3, 3
    q, th, tw = r.standard_normal((BH, H * W, d)), r.standard_normal((2 * H - 1, d)), r.standard_normal((2 * W - 1, d))
    gh, gw = r.standard_normal((BH, H * W, H)), r.standard_normal((BH, H * W, W))

    def loss(q, th, tw):
        rh, rw = oracle.project(q, th, tw, H, W)
        return float((gh * rh).sum() + (gw * rw).sum())

    dq, dth, dtw = oracle.project_backward(q, th, tw, gh, gw, H, W)
    assert near(dq, fd(lambda t: loss(t, th, tw), q))
    assert near(dth, fd(lambda t: loss(q, t, tw), th))
    assert near(dtw, fd(lambda t: loss(q, th, t), tw))
    # the whole chain is the fused backward
    k, v, do = (r.standard_normal((BH, H * W, d)) for _ in range(3))
    want = oracle.fused_backward(q, k, v, th, tw, H, W, 0.5, do)
    rh, rw = oracle.project(q, th, tw, H, W)
    a = oracle.attention_backward(q, k, v, rh, rw, H, W, 0.5, do)
    pq, pth, ptw = oracle.project_backward(q, th, tw, a[3], a[4], H, W)
    for x, y in zip((a[0] + pq, a[1], a[2], pth, ptw), want):
        assert np.allclose(x, y)


def test_no_gradient_along_an_axis_of_length_one():
    """A term that all keys of a row share moves no probability, also where out has been rounded."""
    r = np.random.default_rng(4)
    for H, W in ((1, 5), (5, 1), (1, 1)):
        N = H * W
        q, k, v, do = (r.standard_normal((2, N, 4)) for _ in range(4))
        rh, rw = r.standard_normal((2, N, H)), r.standard_normal((2, N, W))
        out, lse = oracle.masked_attention(q, k, v, rh, rw, H, W, 0.5)
        grads = oracle.attention_backward_from(q, k, v, rh, rw, out.astype(np.float16), lse, do, H, W, 0.5)
        if H == 1:
            assert np.all(grads[3] == 0)
            assert np.allclose(fd(lambda t: float((do * oracle.masked_attention(q, k, v, t, rw, H, W, 0.5)[0]).sum()), rh), 0,
                               atol=1e-8)
        if W == 1:
            assert np.all(grads[4] == 0)
