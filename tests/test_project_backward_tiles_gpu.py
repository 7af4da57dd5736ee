"""project_backward with many tiles a CTA, and the terms that it splits drel into."""
from __future__ import annotations

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


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,H,W", [(64, 24, 21), (128, 9, 35), (64, 40, 40)])
def test_many_tiles_a_cta(d, H, W, dtype):
    """Every CTA takes five tiles at least, so that both buffers of its accumulators are used again, and the last tile
    is cut short.

    drel enters as three bf16 terms, which leave out 2^-24 of a value: nothing next to the sums' own roundings.  The tensor
    core adds 16 rows at a time to what it has and may cut 2^-23 of that off, 2^-24 in the mean and always towards zero, so
    that a tile's sums of n products lose up to n 2^-24 of themselves, and sums over tiles the same share: n = 8 for each product of
    terms (three with bf16, five with fp16) over a tile's 128 tokens, and (2L + 14) / 16 over each table's rows for dq.  (That
    the third term is there shows below, to the last bit.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N = H * W
    BH = 5 * (sms // (d // 64)) * 128 // N + 1
    while BH * N % 128 == 0:
        BH += 1
    g = torch.Generator(device="cuda").manual_seed(H + d)
    q = torch.randn(BH, N, d, generator=g, device="cuda").to(dtype)
    th, tw = (torch.randn(2 * L - 1, d, generator=g, device="cuda").to(dtype) for L in (H, W))
    size = torch.exp(torch.randn(BH, N, 1, generator=g, device="cuda"))
    gh, gw = (size * torch.randn(BH, N, L, generator=g, device="cuda") for L in (H, W))
    base = torch.randn(BH, N, d, generator=g, device="cuda")
    want = oracle.project_backward(*(f64(t) for t in (q, th, tw, gh, gw)), H, W)
    got = rpb.project_backward(q, th, tw, gh, gw, H, W, dq=base)
    terms = 3 if dtype == BF else 5
    steps = ((2 * H + 14) // 16 + (2 * W + 14) // 16, 8, 8)
    for name, a, b, n in zip(("dq", "drel_pos_h", "drel_pos_w"), got, (want[0] + f64(base), *want[1:]), steps):
        rel = np.linalg.norm(f64(a) - b) / np.linalg.norm(b)
        assert rel <= terms * n * 2.0 ** -24, f"{name} {rel:.2e}"
        # no row or column alone is off (a wrong tile would be off by as much as it holds)
        worst = (np.linalg.norm(f64(a) - b, axis=-1) / np.linalg.norm(b, axis=-1)).max()
        assert worst <= 2.0 ** -16, f"{name} {worst:.2e}"
    low = rpb.project_backward(q, th, tw, gh, gw, H, W, dq=base.to(dtype))
    assert torch.equal(low[1], got[1]) and torch.equal(low[2], got[2])
    b = want[0] + f64(base.to(dtype))
    assert np.linalg.norm(f64(low[0]) - b) <= (torch.finfo(dtype).eps / 2 + 2.0 ** -16) * np.linalg.norm(b)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,L", [(64, 8), (128, 8), (128, 11)])
def test_every_bit_of_drel_arrives(d, L, dtype):
    """With unit vectors for q each entry of the tables' gradients is one value of drel, and with unit vectors for the
    tables so is each entry of dq: three bf16 terms hold all 24 bits, so the results are equal."""
    N = L * L
    g = torch.Generator(device="cuda").manual_seed(L)
    gh, gw = (torch.exp(3 * torch.randn(1, N, L, generator=g, device="cuda")) * torch.randn(1, N, L, generator=g, device="cuda")
              for _ in range(2))
    eye = torch.eye(N, d, device="cuda").to(dtype)[None]
    th = torch.zeros(2 * L - 1, d, device="cuda", dtype=dtype)
    tw = th.clone()
    i = torch.arange(2 * L - 1, device="cuda")
    th[i, i], tw[i, i + 32] = 1, 1
    dq, dth, dtw = rpb.project_backward(eye, th, tw, gh, gw, L, L)
    want = [torch.zeros_like(t) for t in (dq, dth, dtw)]
    for n in range(min(N, d)):
        for k in range(L):
            want[1][n // L - k + L - 1, n] = gh[0, n, k]
            want[2][n % L - k + L - 1, n] = gw[0, n, k]
    for n in range(N):
        for k in range(L):
            want[0][0, n, n // L - k + L - 1] = gh[0, n, k]
            want[0][0, n, 32 + n % L - k + L - 1] = gw[0, n, k]
    assert torch.equal(dth, want[1]) and torch.equal(dtw, want[2])
    assert torch.equal(dq, want[0])
