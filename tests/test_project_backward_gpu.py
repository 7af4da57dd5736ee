"""project_backward against the CPU float64 oracle, and a whole training step of the two-step form.

Tolerances.  drel enters the products as three bf16 terms, which leave out at most 2^-24 of a value (two, 2^-16, for a
16-bit dq, and with fp16 q and tables products of small terms, 2^-16, too); the sums are fp32.  A sum over K terms in fp32, in
any order, is off by at most K 2^-24 of the sum of their sizes, and by far less with terms of
either sign; 2^-14 of that sum covers the split and chains of 1000.  dq is rounded once more (eps / 2).
"""
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


def make(BH, H, W, d, dtype, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed)
    N = H * W
    rows = size * torch.exp(torch.randn(BH, N, 1, generator=g))
    x = dict(q=torch.randn(BH, N, d, generator=g).to(dtype), th=torch.randn(2 * H - 1, d, generator=g).to(dtype),
             tw=torch.randn(2 * W - 1, d, generator=g).to(dtype), gh=rows * torch.randn(BH, N, H, generator=g),
             gw=rows * torch.randn(BH, N, W, generator=g), dq=size * torch.randn(BH, N, d, generator=g))
    return {n: t.cuda() for n, t in x.items()}


def check(x, H, W, dq_in, got, what):
    f = {n: f64(t) for n, t in x.items()}
    want = oracle.project_backward(f["q"], f["th"], f["tw"], f["gh"], f["gw"], H, W)
    size = oracle.project_backward(*(np.abs(f[n]) for n in ("q", "th", "tw", "gh", "gw")), H, W)
    base = 0.0 if dq_in is None else f64(dq_in)
    for name, g, ref, tol in zip(("dq", "drel_pos_h", "drel_pos_w"), got, (want[0] + base, *want[1:]), size):
        tol = 2.0 ** -14 * (tol + (np.abs(base) if name == "dq" else 0))
        tol = tol + torch.finfo(g.dtype).eps / 2 * np.abs(ref) + (2.0 ** -25 if g.dtype == HF else 1e-37)
        assert np.isfinite(f64(g)).all(), f"{what} {name}"
        over = (np.abs(f64(g) - ref) - tol).max()
        assert over <= 0, f"{what} {name}: {over:.3e} over its tolerance of up to {tol.max():.3e}"


SIZES = [(1, 1, 1), (3, 1, 5), (2, 5, 1), (5, 14, 14), (2, 16, 16), (3, 7, 30), (1, 40, 40), (2, 64, 2), (2, 2, 64), (1, 64, 64),
         (9, 33, 9), (1, 3, 43), (70, 13, 17)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("BH,H,W", SIZES)
def test_sizes(BH, H, W, d, dtype):
    x = make(BH, H, W, d, dtype, seed=H * 65 + W)
    got = rpb.project_backward(x["q"], x["th"], x["tw"], x["gh"], x["gw"], H, W)
    assert all(g.dtype == FL for g in got)
    check(x, H, W, None, got, f"{BH}x{H}x{W}")
    dq = x["dq"].to(dtype)
    got16 = rpb.project_backward(x["q"], x["th"], x["tw"], x["gh"], x["gw"], H, W, dq=dq)
    assert got16[0].dtype == dtype
    check(x, H, W, dq, got16, f"{BH}x{H}x{W} dq")
    for a, b in zip(got[1:], got16[1:]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("size", [1e-12, 1e10])
def test_gradients_of_any_size(size):
    """fp16 operands, bias gradients far outside fp16's range."""
    x = make(3, 12, 10, 64, HF, seed=3, size=size)
    got = rpb.project_backward(x["q"], x["th"], x["tw"], x["gh"], x["gw"], 12, 10, dq=x["dq"])
    check(x, 12, 10, x["dq"], got, f"size {size}")


def test_many_tiles_streams_and_graph():
    """Several tiles a CTA; the same bits on another stream, in a replayed graph and over a NaN workspace."""
    BH, H, W, d = 30, 32, 32, 64
    x = make(BH, H, W, d, BF, seed=4)
    ws = torch.full((rpb.project_backward_workspace_size(BH, H, W, d) // 4,), float("nan"), device="cuda")

    def step(**more):
        return rpb.project_backward(x["q"], x["th"], x["tw"], x["gh"], x["gw"], H, W, dq=x["dq"], **more)
    want = step()
    check(x, H, W, x["dq"], want, "tiles")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    step(workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(workspace=ws)
    for t in x.values():
        t.mul_(-0.5)
    ws.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(res, step()):
        assert torch.equal(a, b)


def test_in_place_through_the_c_entry():
    """dq_in may be dq itself."""
    x = make(2, 9, 11, 128, BF, seed=5)
    want = rpb.project_backward(x["q"], x["th"], x["tw"], x["gh"], x["gw"], 9, 11, dq=x["dq"])
    dq, dth, dtw = x["dq"].clone(), torch.empty_like(want[1]), torch.empty_like(want[2])
    n = rpb.project_backward_workspace_size(2, 9, 11, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = rpb.load_library().dera_relpos_project_backward(
        x["q"].data_ptr(), x["th"].data_ptr(), x["tw"].data_ptr(), x["gh"].data_ptr(), x["gw"].data_ptr(), dq.data_ptr(),
        dq.data_ptr(), dth.data_ptr(), dtw.data_ptr(), 2, 9, 11, 128, rpb.DERA_BF16, rpb.DERA_F32, ws.data_ptr(), n,
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    for a, b in zip((dq, dth, dtw), want):
        assert torch.equal(a, b)


def test_empty_batch():
    e = torch.empty(0, 6, 64, dtype=BF, device="cuda")
    th, tw = torch.ones(3, 64, dtype=BF, device="cuda"), torch.ones(5, 64, dtype=BF, device="cuda")
    got = rpb.project_backward(e, th, tw, torch.empty(0, 6, 2, device="cuda"), torch.empty(0, 6, 3, device="cuda"), 2, 3)
    assert got[0].shape == (0, 6, 64) and torch.count_nonzero(got[1]) == 0 and torch.count_nonzero(got[2]) == 0


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
def test_training_step(d, dtype):
    """A whole step from the packed projection to its gradient, eager and as a replayed graph, against
    the chain of the oracle's operators on the same intermediate values."""
    B, heads, H, W = 2, 3, 10, 12
    N, BH, scale = H * W, B * heads, d ** -0.5
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(B, N, 3 * heads, d, generator=g).to(dtype).cuda()
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2)]
    ang = torch.randn(N, d // 2, generator=g)
    th, tw = ((0.3 * torch.randn(2 * L - 1, d, generator=g)).to(dtype).cuda() for L in (H, W))
    dout = torch.randn(BH, N, d, generator=g).to(dtype).cuda()
    kw = dict(q_weight=w[0], k_weight=w[1], cos=ang.cos().cuda(), sin=ang.sin().cuda())

    def step():
        q_, k_, v_ = (qkv[:, :, i * heads:(i + 1) * heads] for i in range(3))
        q, k, v = rpb.qk_norm_rope(q_, k_, v_, **kw)
        rh, rw = rpb.project(q, th, tw, H, W)
        out, lse = rpb.attention_lse(q, k, v, rh, rw, H, W, scale)
        dq, dk, dv, drh, drw = rpb.attention_backward(q, k, v, rh, rw, out, lse, dout, H, W, scale)
        dq, dth, dtw = rpb.project_backward(q, th, tw, drh, drw, H, W, dq=dq)
        dqkv = torch.empty_like(qkv)
        parts = [dqkv[:, :, i * heads:(i + 1) * heads] for i in range(3)]
        grads = rpb.qk_norm_rope_backward(q_, k_, dq, dk, dv, dq=parts[0], dk=parts[1], dv=parts[2], **kw)
        return dqkv, dth, dtw, grads[3], grads[4], out, lse, q, k, v

    res = step()
    f = [f64(t) for t in res]
    # the oracle's step, from the same packed projection
    x, c, s = f64(qkv), np.cos(ang.numpy().astype(np.float64)), np.sin(ang.numpy().astype(np.float64))
    xq, xk = x[:, :, :heads], x[:, :, heads:2 * heads]
    q, k, v = f[7], f[8], f[9]
    for name, a, b in (("q", q, oracle.qk_norm_rope(xq, f64(w[0]), c, s)), ("k", k, oracle.qk_norm_rope(xk, f64(w[1]), c, s))):
        assert np.abs(a - b).max() <= torch.finfo(dtype).eps / 2 * np.abs(b).max() * 1.01, name
    want = oracle.fused_backward(q, k, v, f64(th), f64(tw), H, W, scale, f64(dout))
    dxq, dwq = oracle.qk_norm_rope_backward(xq, want[0], f64(w[0]), c, s)
    dxk, dwk = oracle.qk_norm_rope_backward(xk, want[1], f64(w[1]), c, s)
    dxv = want[2].reshape(B, heads, N, d).transpose(0, 2, 1, 3)
    # each gradient passes the roundings of out, P and dZ: relative errors of u in terms that cancel,
    # within 4 u of the gradient's norm (one u from each, and one of the last rounding)
    u = torch.finfo(dtype).eps / 2
    for name, a, b in (("dqkv", f[0], np.concatenate((dxq, dxk, dxv), 2)), ("drel_pos_h", f[1], want[3]),
                       ("drel_pos_w", f[2], want[4]), ("dq_weight", f[3], dwq), ("dk_weight", f[4], dwk)):
        assert np.linalg.norm(a - b) <= 4 * u * np.linalg.norm(b), name
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    qkv.mul_(0.5).add_(0.25)
    dout.mul_(-1.5)
    graph.replay()
    for a, b in zip(cap, step()):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last heads are what a call on them alone gives.

    attention_lse: P is rounded to 11 bits (2^-11 of a value) relative to a running maximum that may differ between the two
    calls, so outputs differ by 2 * 2^-11 of sum P |v| <= max |v| each, and by their own rounding.
    attention_backward, from the same out and lse: sums of 4096 terms in another order where a unit is
    cut, 2 * 4096 * 2^-24 = 2^-11 of the sum of magnitudes, which for independent terms is some sqrt(4096)
    times the result: 2^-5 in norm.  A wrong offset gives 1 or more."""
    if torch.cuda.mem_get_info()[0] < 140e9:
        pytest.skip("needs 140 GB")
    BH, H, W, d = 8200, 64, 64, 64
    N, tail = H * W, slice(BH - 2, BH)
    g = torch.Generator(device="cuda").manual_seed(18)

    def rn(*shape, dtype=BF):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(generator=g)
    q, k, v, do = (rn(BH, N, d) for _ in range(4))
    rh, rw = rn(BH, N, H, dtype=FL), rn(BH, N, W, dtype=FL)
    assert rh.numel() > 2 ** 31 and q.numel() > 2 ** 31
    out, lse = rpb.attention_lse(q, k, v, rh, rw, H, W)
    grads = rpb.attention_backward(q, k, v, rh, rw, out, lse, do, H, W, grad_dtype=BF)
    part = [t[tail].clone() for t in (q, k, v, rh, rw)]
    o2, l2 = rpb.attention_lse(*part, H, W)
    top = part[2].float().abs().max()
    assert (out[tail].float() - o2.float()).abs().max() <= 2 * 2.0 ** -11 * top + 2 * 2.0 ** -8 * o2.float().abs().max()
    assert (lse[tail] - l2).abs().max() <= 2.0 ** -9      # 2 * 2^-11 of the sum, in base 2
    g2 = rpb.attention_backward(*part, out[tail].clone(), lse[tail].clone(), do[tail].clone(), H, W, grad_dtype=BF)
    for a, b in zip(grads, g2):
        assert (a[tail].float() - b.float()).norm() <= (2.0 ** -5 + 2 * 2.0 ** -8) * b.float().norm()
    del k, v, do, rh, rw, out, lse
    th, tw = rn(2 * H - 1, d), rn(2 * W - 1, d)
    dq = rpb.project_backward(q, th, tw, grads[3], grads[4], H, W, dq=grads[0])[0]
    want = rpb.project_backward(q[tail].clone(), th, tw, grads[3][tail].clone(), grads[4][tail].clone(), H, W,
                                dq=grads[0][tail].clone())[0]
    assert torch.equal(dq[tail], want)
    del q, grads, part, g2, dq, want
    torch.cuda.empty_cache()
