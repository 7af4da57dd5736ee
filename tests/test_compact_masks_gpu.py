"""Axes of length one, and biases at the ends of their range, in the compact-bias attention and its backward.

The bias's gradient along an axis of length one is zero by mathematics (the softmax does not see a term that all keys
share), so it is exactly zero.  A bias of -1e38 or below masks its keys, whatever type it has: a call with such values
gives the bits that -inf in their place gives."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu

BF, HF, FL = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()
    yield
    assert rpb.device_status() == 0, "a kernel hit its bounded-wait budget"


def make(BH, H, W, d, dtype, bias, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = H * W
    x = {n: torch.randn(BH, N, d, generator=g, device="cuda").to(dtype) for n in ("q", "k", "v", "dout")}
    x["rel_h"] = (2 * torch.randn(BH, N, H, generator=g, device="cuda")).to(bias)
    x["rel_w"] = (2 * torch.randn(BH, N, W, generator=g, device="cuda")).to(bias)
    return x


def step(x, H, W, **more):
    out, lse = rpb.attention_lse(x["q"], x["k"], x["v"], x["rel_h"], x["rel_w"], H, W, **more)
    grads = rpb.attention_backward(x["q"], x["k"], x["v"], x["rel_h"], x["rel_w"], out, lse, x["dout"], H, W)
    return (out, lse, *grads)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (HF, 128)])
@pytest.mark.parametrize("BH,H,W", [(3, 1, 1), (2, 1, 12), (2, 12, 1), (5, 64, 1), (5, 1, 64), (200, 57, 1)])
def test_axis_of_length_one(BH, H, W, dtype, d):
    x = make(BH, H, W, d, dtype, FL, 100 * H + W)
    grads = step(x, H, W)[2:]
    for L, g in ((H, grads[3]), (W, grads[4])):
        assert torch.count_nonzero(g) == 0 if L == 1 else torch.count_nonzero(g) > 0


@pytest.mark.parametrize("value", [-1e38, -1.7e38, -2.3e38, "half", "lowest"])
@pytest.mark.parametrize("bias", [FL, BF])
@pytest.mark.parametrize("H,W,BH", [(9, 13, 5), (14, 14, 4), (64, 64, 3), (40, 33, 2)])
def test_finite_masks(H, W, BH, bias, value):
    """Some keys by either bias and whole rows by rel_h, in units that are cut (64x64 with a workspace) and whole ones."""
    low = {"half": torch.finfo(bias).min / 2, "lowest": torch.finfo(bias).min}.get(value, value)
    x = make(BH, H, W, 64, BF, bias, 7)
    m = {n: torch.zeros_like(x[n], dtype=torch.bool) for n in ("rel_h", "rel_w")}
    m["rel_h"][:, :, H - 2:] = True
    m["rel_h"][:, 1::5] = True
    m["rel_w"][:, 2::7] = True
    m["rel_w"][:, :, 0] = True
    empty = (m["rel_h"].all(-1) | m["rel_w"].all(-1))
    both = [{**x, **{n: x[n].masked_fill(m[n], to) for n in m}} for to in (low, -math.inf)]
    for workspace in (None, False):
        got, want = (step(b, H, W, workspace=workspace) for b in both)
        for name, a, b in zip(("out", "lse", "dq", "dk", "dv", "drel_h", "drel_w"), got, want):
            assert torch.equal(a, b), f"{name} {workspace}"
        assert torch.count_nonzero(got[0][empty]) == 0 and torch.isneginf(got[1][empty]).all()
        assert torch.isfinite(got[1][~empty]).all()
        assert torch.count_nonzero(got[2][empty]) == 0
    one = [rpb.attention(b["q"], b["k"], b["v"], b["rel_h"], b["rel_w"], H, W) for b in both]
    assert torch.equal(*one)


@pytest.mark.parametrize("low", [-1e4, -1e9, -1e30, 1e9])
@pytest.mark.parametrize("H,W,BH", [(8, 12, 3), (64, 64, 2)])
def test_rows_far_from_zero(H, W, BH, low):
    """A finite bias that all keys of a row share, however large: the softmax does not see it.  Logits spread over some 50
    powers of two.  Every row's out within the forward's bound (2^-11 + 2^-9) max|v| and its own rounding; lse within
    2^-13 and three roundings of fp32 (the shift's conversion to base 2, that constant, and the sum)."""
    x = make(BH, H, W, 64, HF, FL, 8)
    x["q"] = 2.5 * x["q"]
    for n in ("rel_h", "rel_w"):
        y = {m: t.clone() for m, t in x.items()}
        y[n][:, 1::3] = low
        for workspace in (None, False):
            out, lse = rpb.attention_lse(y["q"], y["k"], y["v"], y["rel_h"], y["rel_w"], H, W, 0.25, workspace=workspace)
            f = {m: t.double().cpu().numpy() for m, t in y.items()}
            base = {m: f[m] for m in ("rel_h", "rel_w")}
            base[n] = base[n].copy()
            base[n][:, 1::3] = 0
            want, l0 = oracle.masked_attention(f["q"], f["k"], f["v"], base["rel_h"], base["rel_w"], H, W, 0.25)
            tol = (2.0 ** -11 + 2.0 ** -9) * np.abs(f["v"]).max() + 2.0 ** -11 * np.abs(want)
            got = out.double().cpu().numpy()
            assert np.isfinite(got).all(), n
            assert (np.abs(got - want) <= tol).all(), n
            l0[:, 1::3] += np.float32(low) / math.log(2.0)
            assert (np.abs(lse.double().cpu().numpy() - l0) <= 2.0 ** -13 + 3 * 2.0 ** -24 * np.abs(l0)).all(), n


@pytest.mark.parametrize("low", [-1e9, -1e30])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_beside_rows_far_from_zero(d, low):
    """A row masked as a whole by a finite value whose lse says nothing of its probabilities gives no gradient: the
    others get the bits that they get with -inf there."""
    H, W = 11, 20
    x = make(4, H, W, d, BF, FL, 10)
    for n in ("rel_h", "rel_w"):
        both = []
        for to in (low, -math.inf):
            y = {m: t.clone() for m, t in x.items()}
            y[n][:, 2::5] = to
            both.append(step(y, H, W))
        rest = torch.arange(H * W, device="cuda") % 5 != 2
        for a, b in zip(both[0][:2], both[1][:2]):
            assert torch.equal(a[:, rest], b[:, rest])
        for a, b in zip(both[0][2:], both[1][2:]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bias", [BF, HF])
@pytest.mark.parametrize("BH,H,W", [(3, 1, 1), (5, 3, 7), (3, 13, 13), (3, 15, 9), (7, 35, 35), (3, 63, 63), (5, 63, 64), (3, 64, 61),
                                    (3, 14, 13), (1, 5, 1)])
def test_16_bit_bias_of_any_length(BH, H, W, bias):
    """A 16-bit bias gives the bits of the same values in fp32: rows that start in the middle of a word, a tensor
    that ends in one, tiles behind the last row."""
    x = make(BH, H, W, 64, BF, bias, 9)
    y = {**x, "rel_h": x["rel_h"].float(), "rel_w": x["rel_w"].float()}
    for a, b in zip(step(x, H, W), step(y, H, W)):
        assert torch.equal(a, b)
