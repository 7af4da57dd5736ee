"""Axes of length one, and biases at the ends of their range, in the compact-bias attention and its backward.

The bias's gradient along an axis of length one is zero by mathematics (the softmax does not see a term that all keys
share), so it is exactly zero."""
from __future__ import annotations

import pytest
import torch

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
