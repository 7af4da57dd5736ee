"""A whole encoder block, forward and backward, as a training step runs it: norms, linear layers, the heads' norms and rotation and the
attention of the framework one after another, against the same block in 64 bits by autograd; eager and replayed."""
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


def make(B, H, W, heads, d, width, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    C, N = heads * d, H * W

    def r(*shape, s=1.0):
        return (s * torch.randn(*shape, generator=g)).to(dtype).cuda()

    ang = torch.randn(N, d // 2, generator=g).cuda()
    p = dict(ln1_w=(1 + 0.2 * torch.randn(C, generator=g)).cuda(), ln1_b=(0.2 * torch.randn(C, generator=g)).cuda(),
             ln2_w=(1 + 0.2 * torch.randn(C, generator=g)).cuda(), ln2_b=(0.2 * torch.randn(C, generator=g)).cuda(),
             qkv_w=r(3 * C, C, s=C ** -0.5), qkv_b=r(3 * C, s=0.2), out_w=r(C, C, s=C ** -0.5), out_b=r(C, s=0.2),
             up_w=r(width, C, s=C ** -0.5), up_b=r(width, s=0.2), down_w=r(C, width, s=width ** -0.5), down_b=r(C, s=0.2),
             th=r(2 * H - 1, d, s=0.2), tw=r(2 * W - 1, d, s=0.2), qw=r(d, s=0.2) + 1, kw=r(d, s=0.2) + 1)
    return p, ang.cos(), ang.sin(), r(B, N, C), r(B, N, C)


def forward(p, cos, sin, x, H, W, heads):
    """y and what the backward needs."""
    B, N, C = x.shape
    d = C // heads
    n1, m1, r1 = rpb.layer_norm(x, p["ln1_w"], p["ln1_b"])
    qkv = rpb.linear(n1, p["qkv_w"], p["qkv_b"]).view(B, N, 3, heads, d)
    q, k, v = rpb.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], q_weight=p["qw"], k_weight=p["kw"], cos=cos, sin=sin)
    rel_h, rel_w = rpb.project(q, p["th"], p["tw"], H, W)
    out, lse = rpb.attention_lse(q, k, v, rel_h, rel_w, H, W)
    o = out.view(B, heads, N, d).transpose(1, 2)          # the heads as they lie
    x2 = rpb.linear(o, p["out_w"], p["out_b"], residual=x)
    n2, m2, r2 = rpb.layer_norm(x2, p["ln2_w"], p["ln2_b"])
    h, pre = rpb.linear(n2, p["up_w"], p["up_b"], activation="gelu", keep_pre=True)
    y = rpb.linear(h, p["down_w"], p["down_b"], residual=x2)
    return y, (x, n1, m1, r1, qkv, q, k, v, rel_h, rel_w, out, lse, o, x2, n2, m2, r2, h, pre)


def backward(p, cos, sin, saved, dy, H, W, heads):
    x, n1, m1, r1, qkv, q, k, v, rel_h, rel_w, out, lse, o, x2, n2, m2, r2, h, pre = saved
    B, N, C = x.shape
    t = x.dtype
    g = {}
    dpre, g["down_w"], g["down_b"] = rpb.linear_backward(dy, h, p["down_w"], input_pre=pre, input_activation="gelu", grad_dtype=t)
    dn2, g["up_w"], g["up_b"] = rpb.linear_backward(dpre, n2, p["up_w"], grad_dtype=t)
    dx2, g["ln2_w"], g["ln2_b"] = rpb.layer_norm_backward(dn2, x2, m2, r2, p["ln2_w"], dres=dy, grad_dtype=t)
    do, g["out_w"], g["out_b"] = rpb.linear_backward(dx2, o, p["out_w"], grad_dtype=t)
    assert do.stride() == o.stride()
    dout = do.transpose(1, 2).reshape(out.shape)          # a view: laid out as the attention takes it
    assert dout.data_ptr() == do.data_ptr()
    dq, dk, dv, dh, dw = rpb.attention_backward(q, k, v, rel_h, rel_w, out, lse, dout, H, W, grad_dtype=t)
    dq, g["th"], g["tw"] = rpb.project_backward(q, p["th"], p["tw"], dh, dw, H, W, dq=dq)
    dqkv = torch.empty_like(qkv)
    _, _, _, g["qw"], g["kw"] = rpb.qk_norm_rope_backward(
        qkv[:, :, 0], qkv[:, :, 1], dq, dk, dv, q_weight=p["qw"], k_weight=p["kw"], cos=cos, sin=sin, dq=dqkv[:, :, 0],
        dk=dqkv[:, :, 1], dv=dqkv[:, :, 2], grad_dtype=t)
    dn1, g["qkv_w"], g["qkv_b"] = rpb.linear_backward(dqkv.view(B, N, 3 * C), n1, p["qkv_w"], grad_dtype=t)
    dx, g["ln1_w"], g["ln1_b"] = rpb.layer_norm_backward(dn1, x, m1, r1, p["ln1_w"], dres=dx2, grad_dtype=t)
    g["x"] = dx
    return g


def reference(p, cos, sin, x, dy, H, W, heads):
    """The block's value and gradients in 64 bits."""
    q64 = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    c, s, xx = cos.double().cpu(), sin.double().cpu(), x.double().cpu().requires_grad_()
    B, N, C = x.shape
    d = C // heads
    ln = torch.nn.functional.layer_norm
    qkv = (ln(xx, (C,), q64["ln1_w"], q64["ln1_b"], 1e-6) @ q64["qkv_w"].T + q64["qkv_b"]).view(B, N, 3, heads, d)

    def head(t, w):
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w
        a, b = t[..., :d // 2], t[..., d // 2:]
        cc, ss = c[None, :, None], s[None, :, None]
        return torch.cat((a * cc - b * ss, b * cc + a * ss), -1).transpose(1, 2)

    q, k, v = head(qkv[:, :, 0], q64["qw"]), head(qkv[:, :, 1], q64["kw"]), qkv[:, :, 2].transpose(1, 2)
    iy, ix = torch.arange(N) // W, torch.arange(N) % W
    rh = torch.einsum("bhnd,nkd->bhnk", q, q64["th"][iy[:, None] - torch.arange(H)[None] + H - 1])
    rw = torch.einsum("bhnd,nkd->bhnk", q, q64["tw"][ix[:, None] - torch.arange(W)[None] + W - 1])
    z = q @ k.mT / math.sqrt(d) + (rh[..., None] + rw[..., None, :]).flatten(-2)
    o = (z.softmax(-1) @ v).transpose(1, 2).reshape(B, N, C)
    x2 = xx + o @ q64["out_w"].T + q64["out_b"]
    h = torch.nn.functional.gelu(ln(x2, (C,), q64["ln2_w"], q64["ln2_b"], 1e-6) @ q64["up_w"].T + q64["up_b"])
    y = x2 + h @ q64["down_w"].T + q64["down_b"]
    y.backward(dy.double().cpu())
    return y.detach(), {n: t.grad for n, t in q64.items()} | {"x": xx.grad}


@pytest.mark.parametrize("B,H,W,heads,d,width,dtype", [(2, 14, 14, 4, 64, 640, BF), (1, 9, 13, 2, 128, 520, HF), (1, 20, 20, 2, 64, 256, BF)])
def test_training_step(B, H, W, heads, d, width, dtype):
    p, cos, sin, x, dy = make(B, H, W, heads, d, width, dtype)
    y, saved = forward(p, cos, sin, x, H, W, heads)
    grads = backward(p, cos, sin, saved, dy, H, W, heads)
    wy, wg = reference(p, cos, sin, x, dy, H, W, heads)
    # A dozen roundings to 16 bits lie between the block's input and its output, as many again on the way back: of independent signs they add
    # up to sqrt(24) of one, eps / 2 / sqrt(3) of the root mean square each; four times that.
    tol = 4 * math.sqrt(24) * torch.finfo(dtype).eps / 2 / math.sqrt(3)
    for name, got, want in [("y", y, wy)] + [(n, grads[n], wg[n]) for n in wg]:
        got = got.double().cpu().reshape(want.shape)
        rel = float((got - want).norm() / want.norm())
        assert rel <= tol, f"{name}: {rel:.2e} over {tol:.2e}"
    assert rpb.device_status() == 0


def test_a_captured_step_replays():
    args = (2, 16, 16, 2, 64, 384, BF)
    B, H, W, heads, d, width, dtype = args
    p, cos, sin, x, dy = make(*args)
    y, saved = forward(p, cos, sin, x, H, W, heads)
    want = backward(p, cos, sin, saved, dy, H, W, heads)
    torch.cuda.synchronize()
    xs, dys = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys, ss = forward(p, cos, sin, xs, H, W, heads)
        got = backward(p, cos, sin, ss, dys, H, W, heads)
    for seed in (1, 0):   # other inputs first
        _, _, _, x2, dy2 = make(*args, seed=seed)
        xs.copy_(x2)
        dys.copy_(dy2)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys, y)
    assert all(torch.equal(got[n], want[n]) for n in want)
