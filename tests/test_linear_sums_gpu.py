"""fp32 results of long contractions of one sign, where the cuts of the tensor core's sums towards zero add up.

The tensor core takes 16 products a step.  It cuts each at a quarter of a unit in the last place of the sum so far, and the new sum at a
whole one (seen with one product of 2^20 beside 15 small ones): 5 units at most, 2.5 on average where products have bits enough.  So a
chain of partial sums P_1 < P_2 < ... is off by sum(4 ulp(P_i-1) + ulp(P_i)) / P_n at most, and by half of that on average over many
results: 3.3e-6 after 512 terms of one size, twice that after 1024.  Chains of 512 terms are added with rounding, at most 2^-24 of a
partial sum each, (n + 1) / 2 * 2^-24 for n of them (few tokens add theirs in fewer steps), which cancels on average; and 2^-23 for
the rest.
"""
from __future__ import annotations

import math

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


def one_sign(g, dt, *shape):
    """Of fp16 a product has 22 bits, so that sums are cut from the first on; of bf16 16, and sums up to 1024 are exact."""
    return (1 + 0.1 * torch.rand(*shape, generator=g, device="cuda")).to(dt)


def ulp(v):
    return 2.0 ** (math.floor(math.log2(v)) - 23)


def most_cut():
    """Of a chain of 512 terms, products of 1.05^2 (relative)."""
    P = [16 * i * 1.05 ** 2 for i in range(1, 33)]
    return sum(4 * ulp(p) + ulp(q) for p, q in zip(P, P[1:])) / P[-1]


def check(got, want, terms):
    off = (got.double() - want) / want
    n = -(-terms // 512)
    assert float(off.abs().max()) <= most_cut() + (n + 1) / 2 * 2.0 ** -24 + 2.0 ** -23
    assert abs(float(off.mean())) <= most_cut() / 2, float(off.mean())
    assert rpb.device_status() == 0


# tokens, terms, results a token
SIZES = [(3000, 16384, 264), (1000, 65536, 520),                      # pairs of CTAs
         (9, 16384, 264), (128, 4096, 1032), (9, 32768, 264),         # few tokens: a cluster a tile
         (9, 65536, 264), (128, 40000, 136),
         (9, 16384, 20488), (100, 4096, 32000), (33, 8192, 12000),    # more tiles than clusters at a time
         (200, 16384, 264), (256, 8192, 384), (300, 65536, 136)]      # clusters beyond 128 tokens


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("N,terms,out", SIZES)
def test_forward(N, terms, out, dt):
    g = torch.Generator(device="cuda").manual_seed(31)
    x, w = one_sign(g, dt, N, terms), one_sign(g, dt, out, terms)
    check(rpb.linear(x, w, out_dtype=F32), x.double() @ w.double().T, terms)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("N,terms,out", SIZES)
def test_input_gradient(N, terms, out, dt):
    g = torch.Generator(device="cuda").manual_seed(32)
    dy, w = one_sign(g, dt, N, terms), one_sign(g, dt, terms, out)
    dx = rpb.linear_backward(dy, torch.empty(N, out, device="cuda", dtype=dt), w, weight_grad=False, bias_grad=False)[0]
    check(dx, dy.double() @ w.double(), terms)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("N,K,out", [(16384, 4096, 4096), (65536, 64, 72), (40000, 1000, 2056)])
def test_weight_gradient(N, K, out, dt):
    g = torch.Generator(device="cuda").manual_seed(33)
    x, dy = one_sign(g, dt, N, K), one_sign(g, dt, N, out)
    dw = rpb.linear_backward(dy, x, torch.empty(out, K, device="cuda", dtype=dt), input_grad=False, bias_grad=False)[1]
    check(dw, dy.double().T @ x.double(), N)
