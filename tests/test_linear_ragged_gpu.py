"""Few tokens in several groups of columns, and features that end inside a warp's rows: lanes without a feature take part in every load
that their warp makes as a whole."""
from __future__ import annotations

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild
from test_linear_gpu import check_backward, check_forward, tokens

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


@pytest.mark.parametrize("N", [1, 17, 33, 64, 100, 128])
@pytest.mark.parametrize("K", [8, 64, 136])
@pytest.mark.parametrize("out", [8, 40, 136, 1000])
@pytest.mark.parametrize("dt,od", [(BF, BF), (HF, F32)])
def test_features_inside_a_warp(N, K, out, dt, od):
    g = torch.Generator().manual_seed(21)
    x, w = tokens(1, N, K, 0, dt, g), (torch.randn(out, K, generator=g) * K ** -0.5).to(dt).cuda()
    b, res = torch.randn(out, generator=g).cuda(), torch.randn(1, N, out, generator=g).to(od).cuda()
    y, pre = rpb.linear(x, w, b, activation="gelu", residual=res, keep_pre=True, out_dtype=od)
    check_forward(x, w, y, b, "gelu", res, pre)
    dy, ipre = torch.randn(1, N, out, generator=g).to(dt).cuda(), tokens(1, N, K, 0, dt, g)
    check_backward(dy, x, w, rpb.linear_backward(dy, x, w, input_pre=ipre, input_activation="silu", grad_dtype=od), ipre, "silu")
    assert rpb.device_status() == 0


@pytest.mark.parametrize("N", [150, 600])
@pytest.mark.parametrize("K,out", [(64, 40), (200, 104), (768, 296), (520, 2088)])
@pytest.mark.parametrize("od", [BF, F32])
def test_columns_inside_a_box(N, K, out, od):
    """Tiles whose last columns end inside a box, so that a warp stores one half and not the other."""
    g = torch.Generator().manual_seed(22)
    x, w = tokens(1, N, K, 0, BF, g), (torch.randn(out, K, generator=g) * K ** -0.5).to(BF).cuda()
    b = torch.randn(out, generator=g).cuda()
    y, pre = rpb.linear(x, w, b, activation="gelu", keep_pre=True, out_dtype=od)
    check_forward(x, w, y, b, "gelu", None, pre)
    dy, ipre = torch.randn(1, N, out, generator=g).to(BF).cuda(), tokens(1, N, K, 0, BF, g)
    check_backward(dy, x, w, rpb.linear_backward(dy, x, w, input_pre=ipre, input_activation="gelu", grad_dtype=od), ipre, "gelu")
    assert rpb.device_status() == 0
