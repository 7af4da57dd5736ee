"""qk_norm_rope on rows with infinities past the rotation, and its weight gradients where a block takes several heads."""
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


# heads a block: as many as leave eight blocks an SM; here 4 to 16, and head counts that are no multiple of it
WEIGHT_CASES = [(4, 4096, 7, 5, 64, BF), (2, 4096, 7, 5, 128, HF), (8, 4096, 13, 6, 64, HF), (1, 2, 16384, 37, 64, BF),
                (3, 8190, 9, 3, 128, BF)]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("B,N,hq,hk,d,dtype", WEIGHT_CASES)
def test_weight_gradients_of_many_heads(B, N, hq, hk, d, dtype, fp32):
    """dq_weight and dk_weight against float64 sums over every row.

    A column's sum of R terms is a chain of at most L = R / (partial rows) additions a lane, 5 + 8 more within a block and
    2 * 32 more over the partial rows' sums; each rounds by 2^-24 of a partial sum, no more than the terms' sizes together:
    (L + 128) 2^-24 of their sum bounds it.  The chain of a lane is its tokens times its heads, less than 1024 here, and
    a term itself is off by 16 roundings and the reciprocal root's 2^-22."""
    g = torch.Generator(device="cuda").manual_seed(B * N + hq)
    q, k = (torch.randn(B, N, h, d, generator=g, device="cuda").to(dtype) for h in (hq, hk))
    dz = [torch.randn(B * h, N, d, generator=g, device="cuda") for h in (hq, hk)]
    dz = dz if fp32 else [t.to(dtype) for t in dz]
    ang = torch.randn(N, d // 2, generator=g, device="cuda")
    w = [1 + 0.3 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    got = rpb.qk_norm_rope_backward(q, k, *dz, q_weight=w[0], k_weight=w[1], cos=ang.cos(), sin=ang.sin())
    c, s = ang.cos().double()[:, None], ang.sin().double()[:, None]
    for x, z, dw, dx, wi in ((q, dz[0], got[3], got[0], w[0]), (k, dz[1], got[4], got[1], w[1])):
        h = x.shape[2]
        y = z.view(B, h, N, d).transpose(1, 2).double()
        a, b = y[..., :d // 2], y[..., d // 2:]
        back = torch.cat((a * c + b * s, b * c - a * s), -1)
        xd = x.double()
        r = (xd.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        terms = back * xd * r
        assert ((dw.double() - terms.sum((0, 1, 2))).abs() <= 1200 * 2.0 ** -24 * terms.abs().sum((0, 1, 2))).all()
        # a row counted twice or left out is far outside: its term against the sum's random error
        err = (dw.double() - terms.sum((0, 1, 2))).norm() / terms.square().sum((0, 1, 2)).sqrt().norm()
        assert err <= 2.0 ** -10
        gy = back * wi.double()
        want = r * (gy - xd * r * r * (gy * xd).mean(-1, keepdim=True))
        assert (dx.double() - want).norm() <= 2.0 ** -18 * want.norm()
