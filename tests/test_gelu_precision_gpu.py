"""What include/dera_block.h says of gelu's Phi: off by 2^-18 + u^2 2^-23 of its distance to 0 or 1.

Phi(-z) = exp(-z^2 / 2) t P(t): the fit is 0.94 * 2^-20 off; t (a reciprocal of a product of two sums, a product) 5 * 2^-24, which t P(t)
doubles at most; P's steps 3 * 2^-24 and two products; the exponential 2^-22: 2.2 * 2^-20 together.  The exponential's argument is rounded
three times, 3 * 2^-24 of z^2 / 2.  The result itself is one more rounding.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import relative_position_bias_gb300 as rpb
from block_tolerance import f64
from oracle import block_oracle as ob
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


@pytest.mark.parametrize("N", [3, 200])
@pytest.mark.parametrize("seed", range(4))
def test_phi(N, seed):
    g = torch.Generator().manual_seed(41 + seed)
    u = (26 * torch.rand(4096, generator=g) - 13).cuda()   # past 13 Phi(-z) is below the smallest normal number
    zero = torch.zeros(4096, 8, device="cuda", dtype=torch.bfloat16)
    y = rpb.linear(zero[:N], zero, u, activation="gelu", out_dtype=torch.float32)
    u64, got = f64(u), f64(y)
    want = ob.activation(u64, "gelu")
    tail = np.abs(ob.activation(-np.abs(u64), "gelu"))   # |u| times Phi's distance to 0 or 1
    assert (np.abs(got - want) <= tail * (2.0 ** -18 + u64 ** 2 * 2.0 ** -23) + 2.0 ** -24 * np.abs(want)).all()
