"""qk_norm_rope on rows with infinities past the rotation."""
from __future__ import annotations

import math

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (128, 64), (64, 0)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_elements_past_the_rotation_pass(d, rot, inter, dtype):
    """Without a norm the elements from rotary_dim on are moved bit for bit, infinities and negative zeros among
    them (a NaN stays one), and a rotated element sees its pair alone."""
    B, N, h = 2, 11, 3
    g = torch.Generator().manual_seed(d + rot)
    x = torch.randn(B, N, h, d, generator=g).to(dtype)
    plain = x.clone()
    for n, (at, v) in enumerate(((rot, math.inf), (d - 1, -math.inf), (rot + 3, math.nan), (rot + 2, -0.0), (d - 8, math.inf))):
        x[:, n, :, at] = v
    x, plain = x.cuda(), plain.cuda()
    ang = torch.randn(N, rot // 2, generator=g).cuda() if rot else None
    kw = dict(interleaved=inter, **(dict(cos=ang.cos(), sin=ang.sin()) if rot else {}))

    def same(a, b):
        a, b = a.contiguous(), b.contiguous()
        return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.view(torch.int16)[~a.isnan()], b.view(torch.int16)[~b.isnan()])

    for got, ref in zip(rpb.qk_norm_rope(x, x, **kw), rpb.qk_norm_rope(plain, plain, **kw)):
        moved = got.view(B, h, N, d).transpose(1, 2)
        assert same(moved[..., rot:], x[..., rot:])
        assert torch.equal(got[..., :rot], ref[..., :rot])
    dz = x.transpose(1, 2).reshape(B * h, N, d).contiguous()
    pz = plain.transpose(1, 2).reshape(B * h, N, d).contiguous()
    got = rpb.qk_norm_rope_backward(x, x, dz, dz, grad_dtype=dtype, **kw)
    ref = rpb.qk_norm_rope_backward(plain, plain, pz, pz, grad_dtype=dtype, **kw)
    for a, b in zip(got[:2], ref[:2]):
        assert same(a[..., rot:], x[..., rot:])
        assert torch.equal(a[..., :rot], b[..., :rot])


@pytest.mark.parametrize("inter", [False, True])
def test_infinite_gradient_stays_in_its_column(inter):
    """With a norm, an infinite gradient past the rotation reaches its own column of the weights' gradient and no other."""
    B, N, h, d, rot = 1, 9, 2, 64, 32
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, N, h, d, generator=g).to(BF).cuda()
    dz = torch.randn(B * h, N, d, generator=g).to(BF).cuda()
    ang = torch.randn(N, rot // 2, generator=g).cuda()
    w = torch.ones(d, dtype=BF, device="cuda")
    kw = dict(q_weight=w, k_weight=w, cos=ang.cos(), sin=ang.sin(), interleaved=inter)
    ref = rpb.qk_norm_rope_backward(x, x, dz, dz, **kw)
    bad = dz.clone()
    bad[:, 4, 41] = math.inf
    got = rpb.qk_norm_rope_backward(x, x, bad, bad, **kw)
    keep = torch.arange(d, device="cuda") != 41
    for a, b in zip(got[3:], ref[3:]):
        assert torch.equal(a[keep], b[keep]) and not torch.isfinite(a[41])
