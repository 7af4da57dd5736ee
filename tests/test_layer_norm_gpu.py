"""layer_norm and its backward against the float64 oracle.

Tolerances: every sum over a row is a tree of at most 13 + 16 additions in fp32 (16384 columns: 16 a thread, then lanes and
warps), 32 roundings of 2^-24 with those of the terms: 2^-19 of the sum of the sizes, taken as 2^-18 with the reciprocal
square root's 2^-22 and the last few operations.  A column's sum over rows is 2^-18 of the sum of the sizes for chains of up to
64 additions, which no case here passes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import relative_position_bias_gb300 as rpb
from block_tolerance import f64, near, rounding
from oracle import block_oracle as ob
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TINY = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


def make(rows, C, xd, yd, affine=True, wd=F32, res=False, far=0.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, C, generator=g) * torch.exp(0.5 * torch.randn(C, generator=g)) + 0.5 + far).to(xd).cuda()
    w = (1 + 0.3 * torch.randn(C, generator=g)).to(wd).cuda() if affine else None
    b = torch.randn(C, generator=g).to(wd).cuda() if affine else None
    dy = torch.randn(rows, C, generator=g).to(yd).cuda()
    dres = torch.randn(rows, C, generator=g).to(xd).cuda() if res else None
    return x, w, b, dy, dres


def check_forward(x, w, b, got, eps=1e-6, out=None):
    y, mean, rstd = got
    x64, w64, b64 = f64(x), f64(w), f64(b)
    wy, wm, wr = ob.layer_norm(x64, w64, b64, eps)
    dm = TINY * np.abs(x64).mean(-1)          # of the mean
    near(mean, wm, dm, "mean")
    dr = wr * (TINY + 0.5 * wr * wr * dm * dm)   # of rstd: a mean off by dm adds dm^2 to the variance
    near(rstd, wr, dr, "rstd")
    ww = np.ones(x.shape[-1]) if w64 is None else np.abs(w64)
    xc = np.abs(x64 - wm[..., None])
    size = ww * (wr[..., None] * (dm[..., None] + TINY * xc) + dr[..., None] * xc)
    near(y, wy, rounding(wy, y.dtype) + size + (0 if b64 is None else TINY * np.abs(b64)), "y")


def check_backward(dy, x, mean, rstd, w, dres, got):
    d64, x64, m64, r64, w64 = (f64(t) for t in (dy, x, mean, rstd, w))
    dx, dw, db = ob.layer_norm_backward(d64, x64, m64, r64, w64, f64(dres))
    h = np.abs((x64 - m64[..., None]) * r64[..., None])
    g = np.abs(d64 if w64 is None else d64 * w64)
    size = r64[..., None] * (g + g.mean(-1, keepdims=True) + h * (g * h).mean(-1, keepdims=True))
    if dres is not None:
        size = size + np.abs(f64(dres))
    near(got[0], dx, rounding(dx, got[0].dtype) + TINY * size, "dx")
    if w is None:
        assert got[1] is None and got[2] is None
        return
    axes = tuple(range(x.dim() - 1))
    near(got[1], dw, rounding(dw, F32) + TINY * (np.abs(d64) * h).sum(axes), "dweight")
    near(got[2], db, rounding(db, F32) + TINY * np.abs(d64).sum(axes), "dbias")


CASES = {
    # rows, C, x, y (and dy), affine, weights' type, residual gradient
    "token": (1, 64, BF, BF, True, F32, False),
    "one": (1, 1, F32, F32, True, F32, True),
    "column": (5, 1, HF, HF, True, HF, False),
    "odd": (3, 7, BF, BF, True, BF, True),
    "odd_long": (9, 1001, HF, F32, True, F32, True),
    "eight": (33, 8, HF, HF, True, HF, False),
    "grid12": (196, 768, BF, BF, True, F32, True),
    "stream": (50, 1024, F32, BF, True, F32, True),
    "stream_half": (50, 1000, F32, HF, True, HF, False),
    "plain": (17, 520, BF, F32, False, F32, True),
    "two_k": (31, 2048, HF, HF, True, HF, True),
    "past_two_k": (11, 2056, BF, BF, True, BF, False),
    "odd_past_two_k": (4, 4099, F32, F32, True, F32, True),
    "eight_k": (5, 8192, BF, BF, True, F32, True),
    "longest": (3, 16384, F32, F32, True, F32, True),
    "longest_half": (3, 16384, HF, HF, True, HF, False),
    "odd_longest": (2, 16383, BF, BF, True, F32, False),
    "many": (3000, 96, BF, BF, True, F32, False),
    "many_odd": (2500, 33, HF, HF, True, F32, True),
    "many_wide": (2600, 1536, BF, BF, True, F32, False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_layer_norm(name):
    rows, C, xd, yd, affine, wd, res = CASES[name]
    x, w, b, dy, dres = make(rows, C, xd, yd, affine, wd, res)
    got = rpb.layer_norm(x, w, b, out_dtype=yd)
    assert got[0].dtype == yd
    check_forward(x, w, b, got)
    grads = rpb.layer_norm_backward(dy, x, got[1], got[2], w, dres=dres, grad_dtype=xd)
    assert grads[0].dtype == xd
    check_backward(dy, x, got[1], got[2], w, dres, grads)
    again = rpb.layer_norm_backward(dy, x, got[1], got[2], w, dres=dres, grad_dtype=xd)
    assert all(torch.equal(p, q) for p, q in zip(grads, again) if p is not None)


def test_rows_far_from_zero():
    x, w, b, dy, _ = make(40, 512, F32, F32, far=1000.0)
    got = rpb.layer_norm(x, w, b)
    check_forward(x, w, b, got)
    check_backward(dy, x, got[1], got[2], w, None, rpb.layer_norm_backward(dy, x, got[1], got[2], w))


def test_constant_rows_and_eps():
    x = torch.full((4, 256), 3.0, device="cuda", dtype=HF)
    w = torch.ones(256, device="cuda")
    b = torch.linspace(-1, 1, 256, device="cuda")
    y, mean, rstd = rpb.layer_norm(x, w, b, eps=1e-2, out_dtype=F32)
    assert torch.equal(y, b.expand(4, -1)) and torch.equal(mean, torch.full((4,), 3.0, device="cuda"))
    assert torch.allclose(rstd, torch.full((4,), 10.0, device="cuda"), rtol=1e-6)


@pytest.mark.parametrize("C", [96, 768, 1001, 4096])
def test_infinities_stay_in_their_rows(C):
    x, w, b, dy, _ = make(9, C, BF, BF)
    clean = rpb.layer_norm(x, w, b)
    bad = x.clone()
    bad[2, C // 2], bad[5, C - 1] = float("inf"), float("nan")
    got = rpb.layer_norm(bad, w, b)
    for r in range(9):
        if r in (2, 5):
            assert got[0][r].isnan().all() and got[2][r].isnan()
        else:
            assert all(torch.equal(p[r], q[r]) for p, q in zip(got, clean))


@pytest.mark.parametrize("C,wide", [(256, 512), (256, 264), (64, 71), (33, 40)])
def test_rows_at_a_stride(C, wide):
    x, w, b, dy, _ = make(21, wide, HF, HF)
    x, w, b, dy = x[:, :C], w[:C].contiguous(), b[:C].contiguous(), dy[:, :C].contiguous()
    got = rpb.layer_norm(x, w, b)
    check_forward(x, w, b, got)
    check_backward(dy, x, got[1], got[2], w, None, rpb.layer_norm_backward(dy, x, got[1], got[2], w))


def test_addresses_off_sixteen_bytes():
    """Rows that start at any element: the values are the same."""
    x, w, b, dy, _ = make(6, 64, BF, BF)
    buf = torch.zeros(6 * 64 + 3, dtype=BF, device="cuda")
    off = buf[3:].view(6, 64)
    off.copy_(x)
    want = rpb.layer_norm(x, w, b)
    check_forward(off, w, b, rpb.layer_norm(off, w, b))
    got = rpb.layer_norm_backward(dy, off, want[1], want[2], w)
    check_backward(dy, off, want[1], want[2], w, None, got)


def test_more_dimensions_and_default_types():
    x, w, b, dy, _ = make(24, 128, BF, BF)
    x, dy = x.view(2, 3, 4, 128), dy.view(2, 3, 4, 128)
    y, mean, rstd = rpb.layer_norm(x, w, b)
    assert y.shape == x.shape and y.dtype == BF and mean.shape == rstd.shape == (2, 3, 4)
    dx, dw, db = rpb.layer_norm_backward(dy, x, mean, rstd, w)
    assert dx.shape == x.shape and dx.dtype == dw.dtype == db.dtype == F32
    check_backward(dy, x, mean, rstd, w, None, (dx, dw, db))
    t = x.transpose(0, 1)[:, :1]      # [3, 1, 4, 128]: rows at one stride all the same
    assert torch.equal(rpb.layer_norm(t, w, b)[0], y.transpose(0, 1)[:, :1])
    with pytest.raises(ValueError):
        rpb.layer_norm(x.transpose(0, 1), w, b)


def test_no_rows():
    x = torch.zeros(0, 64, device="cuda", dtype=BF)
    w = torch.ones(64, device="cuda")
    y, mean, rstd = rpb.layer_norm(x, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = rpb.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_streams_and_graphs():
    x, w, b, dy, dres = make(300, 384, BF, BF, res=True)
    want = rpb.layer_norm(x, w, b)
    wantg = rpb.layer_norm_backward(dy, x, want[1], want[2], w, dres=dres, grad_dtype=BF)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = rpb.layer_norm(x, w, b, stream=side)
    gotg = rpb.layer_norm_backward(dy, x, got[1], got[2], w, dres=dres, grad_dtype=BF, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*want, *wantg), (*got, *gotg)))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = rpb.layer_norm(x, w, b)
            outs.append((*o, *rpb.layer_norm_backward(dy, x, o[1], o[2], w, dres=dres, grad_dtype=BF)))
        graphs.append(g)
    s2 = torch.cuda.Stream()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip((*want, *wantg), o))


def test_workspaces():
    x, w, b, dy, _ = make(900, 264, BF, BF)
    _, mean, rstd = rpb.layer_norm(x, w, b)
    need = rpb.layer_norm_backward_workspace_size(900, 264)
    ws = torch.full((need + 16,), 0xff, dtype=torch.uint8, device="cuda")
    want = rpb.layer_norm_backward(dy, x, mean, rstd, w)
    got = rpb.layer_norm_backward(dy, x, mean, rstd, w, workspace=ws[:need])
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and (ws[need:] == 0xff).all()
    for bad, status in ((ws[:need - 256], 9), (ws[16:], 5)):
        with pytest.raises(rpb.DeraError) as e:
            rpb.layer_norm_backward(dy, x, mean, rstd, w, workspace=bad)
        assert e.value.status == status
    assert rpb.device_status() == 0


def test_more_than_two_to_the_31_elements():
    rows, C = (1 << 31) // 2048 + 5, 2048
    x = torch.empty(rows, C, device="cuda", dtype=BF)
    x[:-8] = 0
    tail = torch.randn(8, C, device="cuda").to(BF)
    x[-8:] = tail
    w = 1 + 0.2 * torch.randn(C, device="cuda")
    y, mean, rstd = rpb.layer_norm(x, w)
    y2, mean2, rstd2 = rpb.layer_norm(tail, w)
    assert torch.equal(y[-8:], y2) and torch.equal(mean[-8:], mean2) and torch.equal(rstd[-8:], rstd2)
    dx, dw, _ = rpb.layer_norm_backward(y, x, mean, rstd, w, grad_dtype=BF)
    dx2, dw2, _ = rpb.layer_norm_backward(y2, tail, mean2, rstd2, w, grad_dtype=BF)
    assert torch.equal(dx[-8:], dx2) and torch.allclose(dw, dw2, rtol=1e-5, atol=1e-4)
