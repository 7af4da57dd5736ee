"""layer_norm_backward where mean * rstd is past fp32: what lies past a row's end, and rows that a block does not have, are no part
of any sum.  Tolerances as in test_layer_norm_gpu."""
from __future__ import annotations

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild
from test_layer_norm_gpu import check_backward

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,C", [(1, 96), (9, 96), (5, 97), (3, 8), (4, 520), (3, 1001), (2, 2056), (3, 4099), (2, 8200), (2, 8201),
                                    # more rows than the blocks take at a time, and not a whole number of sets
                                    (5001, 96), (5001, 256), (5003, 33), (3001, 520), (3003, 257)])
def test_large_constant_rows(rows, C, dt):
    """Of 2^112, a power of two: the rows' deviations are exactly zero, while mean * rstd is 5e39 with eps = 1e-12."""
    g = torch.Generator().manual_seed(3)
    big = 2.0 ** 112
    x = torch.full((rows, C), big, dtype=dt, device="cuda")
    mean = torch.full((rows,), big, device="cuda")
    rstd = torch.full((rows,), 1e6, device="cuda")
    w = (1 + 0.3 * torch.randn(C, generator=g)).cuda()
    dy = torch.randn(rows, C, generator=g).to(dt).cuda()
    got = rpb.layer_norm_backward(dy, x, mean, rstd, w)
    check_backward(dy, x, mean, rstd, w, None, got)
    assert not got[1].any()


def test_the_forward_gives_such_statistics():
    x = torch.full((7, 96), 2.0 ** 119, dtype=BF, device="cuda")
    w = torch.ones(96, device="cuda")
    y, mean, rstd = rpb.layer_norm(x, w)
    assert not y.any() and (mean == 2.0 ** 119).all() and torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    dy = torch.randn(7, 96, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    check_backward(dy, x, mean, rstd, w, None, rpb.layer_norm_backward(dy, x, mean, rstd, w))
