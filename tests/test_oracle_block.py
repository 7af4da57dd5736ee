"""The block's float64 oracle against PyTorch's autograd in 64 bits and against differences."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import block_oracle as ob

ACTS = [None, "relu", "gelu", "gelu_tanh", "quick_gelu", "silu"]


def _t(x):
    return torch.from_numpy(x).requires_grad_()


def _act(u, act):
    if act is None:
        return u
    if act == "quick_gelu":
        return u * torch.sigmoid(1.702 * u)
    if act == "gelu_tanh":
        return torch.nn.functional.gelu(u, approximate="tanh")
    return {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[act](u)


@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 5, 16)])
@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm(shape, affine):
    r = np.random.default_rng(0)
    x, dy, C = r.standard_normal(shape) + 3, r.standard_normal(shape), shape[-1]
    w, b = (r.standard_normal(C), r.standard_normal(C)) if affine else (None, None)
    y, mean, rstd = ob.layer_norm(x, w, b, 1e-5)
    xt = _t(x)
    wt, bt = (_t(w), _t(b)) if affine else (None, None)
    yt = torch.nn.functional.layer_norm(xt, (C,), wt, bt, 1e-5)
    assert np.allclose(y, yt.detach().numpy(), rtol=1e-11, atol=1e-11)
    yt.backward(torch.from_numpy(dy))
    dx, dw, db = ob.layer_norm_backward(dy, x, mean, rstd, w, dres=dy)
    assert np.allclose(dx - dy, xt.grad.numpy(), rtol=1e-9, atol=1e-10)
    if affine:
        assert np.allclose(dw, wt.grad.numpy()) and np.allclose(db, bt.grad.numpy())


@pytest.mark.parametrize("act", ACTS)
def test_activation(act):
    u = np.concatenate([np.linspace(-9, 9, 401), [-30.0, 30.0]]) + 1e-3
    assert np.allclose(ob.activation(u, act), _act(torch.from_numpy(u), act).numpy(), rtol=1e-11, atol=1e-14)
    h = 1e-6
    diff = (ob.activation(u + h, act) - ob.activation(u - h, act)) / (2 * h)
    assert np.abs(diff - ob.activation_slope(u, act)).max() < 1e-8


@pytest.mark.parametrize("act", ACTS)
def test_linear(act):
    r = np.random.default_rng(1)
    pre, w, b, dy = (r.standard_normal(s) for s in ((5, 8), (16, 8), (16,), (5, 16)))
    pt, wt, bt = _t(pre), _t(w), _t(b)
    yt = _act(pt, act) @ wt.T + bt
    yt.backward(torch.from_numpy(dy))
    x = ob.activation(pre, act)
    y, u = ob.linear(x, w, b)
    assert np.allclose(y, yt.detach().numpy()) and np.array_equal(y, u)
    dx, dw, db = ob.linear_backward(dy, x, w, pre if act else None, act)
    for got, want in ((dx, pt), (dw, wt), (db, bt)):
        assert np.allclose(got, want.grad.numpy(), rtol=1e-10, atol=1e-12)
    y2, u2 = ob.linear(x, w, b, act, residual=dy)
    assert np.allclose(y2, ob.activation(u2, act) + dy)
