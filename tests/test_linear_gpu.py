"""linear, linear_backward and activation_backward against the float64 oracle (tolerances: block_tolerance)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_tolerance as tol
import relative_position_bias_gb300 as rpb
from block_tolerance import f64, near, rounding
from oracle import block_oracle as ob
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = [None, "relu", "gelu", "gelu_tanh", "quick_gelu", "silu"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


def tokens(B, N, K, d, dtype, g):
    """[B, N, K], or with d [B, N, heads, d] over [B * heads, N, d]."""
    if d:
        return torch.randn(B * (K // d), N, d, generator=g).to(dtype).cuda().view(B, K // d, N, d).transpose(1, 2)
    return torch.randn(B, N, K, generator=g).to(dtype).cuda()


def flat(t, K):
    return f64(t).reshape(-1, K)


def check_forward(x, w, got, bias=None, act=None, residual=None, pre=None):
    out, K = w.shape
    x64, w64 = flat(x, K), f64(w)
    y, u = ob.linear(x64, w64, f64(bias), act, None if residual is None else flat(residual, out))
    du = tol.product(x64, w64) + (0 if bias is None else 2.0 ** -23 * np.abs(f64(bias))) + 2.0 ** -23 * np.abs(u)
    assert got.shape == (x.shape[0], x.shape[1], out)
    # no activation here is steeper than 1.13
    dy = 1.13 * du + tol.act(u, act) + (0 if residual is None else 2.0 ** -23 * np.abs(y))
    near(got.reshape(-1, out), y, rounding(y, got.dtype) + dy, "y")
    if pre is not None:
        near(pre.reshape(-1, out), u, rounding(u, pre.dtype) + du, "pre")


def check_backward(dy, x, w, got, pre=None, act=None):
    out, K = w.shape
    g64, x64, w64 = flat(dy, out), flat(x, K), f64(w)
    p64 = None if pre is None else flat(pre, K)
    dx, dw, db = ob.linear_backward(g64, x64, w64, p64, act)
    if got[0] is not None:
        d = tol.product(g64, w64.T)
        if pre is not None:
            d = d * np.abs(ob.activation_slope(p64, act)) + np.abs(g64 @ w64) * tol.slope(p64, act)
        assert got[0].shape == x.shape
        near(got[0].reshape(-1, K), dx, rounding(dx, got[0].dtype) + d + 2.0 ** -23 * np.abs(dx), "dx")
    if got[1] is not None:
        near(got[1], dw, rounding(dw, got[1].dtype) + tol.product(g64.T, x64.T), "dweight")
    if got[2] is not None:
        near(got[2], db, rounding(db, F32) + 2.0 ** -18 * np.abs(g64).sum(0), "dbias")


SIZES = {
    # B, N, K, out, head_dim (0: rows), dtype, out / grad dtype
    "smallest": (1, 1, 8, 8, 0, BF, BF),
    "token": (1, 1, 1024, 4096, 0, BF, BF),
    "tokens": (32, 1, 768, 264, 0, HF, F32),
    "tokens_heads": (5, 1, 256, 72, 64, BF, BF),
    "thirty_three": (1, 33, 200, 136, 0, HF, HF),
    "long_contraction": (1, 17, 4096, 520, 0, BF, BF),
    "odd_pieces": (3, 40, 1096, 264, 0, HF, HF),
    "few_heads_long": (1, 70, 2304, 72, 128, BF, F32),
    "sixty_five": (5, 13, 640, 1000, 0, BF, F32),
    "tile": (1, 128, 64, 128, 0, BF, BF),
    "past_a_tile": (1, 129, 72, 136, 0, BF, BF),
    "batches": (2, 130, 200, 264, 0, HF, HF),
    "narrow": (1, 300, 1000, 8, 0, BF, BF),
    "window": (3, 196, 768, 776, 0, BF, BF),
    "heads": (2, 196, 384, 520, 64, BF, BF),
    "heads128": (3, 70, 384, 256, 128, HF, F32),
    "heads_few": (2, 5, 128, 40, 64, HF, HF),
    "heads_one": (2, 300, 64, 64, 64, BF, BF),
    "long": (1, 200, 4104, 328, 0, BF, F32),
    "many_features": (1, 32, 768, 2088, 0, HF, F32),
    "long_tiles": (1, 600, 3144, 456, 0, HF, HF),
    "long_heads": (1, 257, 4096, 264, 64, BF, F32),
    "long_gradient": (2, 150, 264, 4104, 0, BF, F32),
    "wide": (1, 260, 136, 2304, 0, HF, HF),
    "image": (1, 1369, 256, 520, 0, BF, F32),
    "pairs": (1, 2500, 200, 2056, 0, BF, BF),
    "pairs_heads": (3, 700, 384, 2000, 64, HF, HF),
    "pairs_narrow": (2, 4900, 320, 136, 0, BF, F32),
    "pairs_many_tiles": (1, 10000, 264, 1032, 0, HF, HF),
    "pairs_wide_f32": (1, 10000, 200, 1032, 0, BF, F32),
    "pairs_wide_heads": (3, 3000, 384, 1096, 64, BF, BF),
    "pairs_wide_heads_f32": (2, 5000, 320, 1064, 64, HF, F32),
}


@pytest.mark.parametrize("name", list(SIZES))
def test_sizes(name):
    B, N, K, out, d, dt, od = SIZES[name]
    g = torch.Generator().manual_seed(1)
    x = tokens(B, N, K, d, dt, g)
    w = (torch.randn(out, K, generator=g) * K ** -0.5).to(dt).cuda()
    b = torch.randn(out, generator=g).to(dt).cuda()
    res = torch.randn(B, N, out, generator=g).to(od).cuda()
    y, pre = rpb.linear(x, w, b, activation="gelu", residual=res, keep_pre=True, out_dtype=od)
    assert y.dtype == od and pre.dtype == dt
    check_forward(x, w, y, b, "gelu", res, pre)
    check_forward(x, w, rpb.linear(x, w))
    check_forward(x, w, rpb.linear(x, w, b.float(), residual=res, out_dtype=od), b, None, res)
    y, pre = rpb.linear(x, w, b, activation="silu", keep_pre=True, out_dtype=od)
    check_forward(x, w, y, b, "silu", None, pre)
    dy = torch.randn(B, N, out, generator=g).to(dt).cuda()
    got = rpb.linear_backward(dy, x, w, grad_dtype=od)
    assert got[0].dtype == od and got[1].dtype == got[2].dtype == F32
    if d and K > d:
        assert got[0].stride() == x.stride()
    check_backward(dy, x, w, got)
    ipre = tokens(B, N, K, d, dt, g)
    got2 = rpb.linear_backward(dy, x, w, input_pre=ipre, input_activation="gelu", weight_grad_dtype=dt)
    assert got2[0].dtype == F32 and got2[1].dtype == dt
    check_backward(dy, x, w, got2, ipre, "gelu")
    got3 = rpb.linear_backward(dy, x, w, input_pre=ipre, input_activation="relu", grad_dtype=od, weight_grad=False)
    check_backward(dy, x, w, got3, ipre, "relu")
    got4 = rpb.linear_backward(dy, x, w, input_pre=ipre, input_activation="gelu", grad_dtype=dt, weight_grad=False)
    check_backward(dy, x, w, got4, ipre, "gelu")
    again = rpb.linear_backward(dy, x, w, grad_dtype=od)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    assert rpb.device_status() == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [7, 150])
def test_activations(act, N):
    g = torch.Generator().manual_seed(2)
    x, w = tokens(1, N, 96, 0, BF, g), (0.4 * torch.randn(104, 96, generator=g)).to(BF).cuda()
    b = torch.randn(104, generator=g).cuda()
    for od in (BF, F32):
        y, pre = rpb.linear(x, w, b, activation=act, keep_pre=True, out_dtype=od)
        check_forward(x, w, y, b, act, None, pre)
    dy = torch.randn(1, N, 104, generator=g).to(BF).cuda()
    if act:
        ipre = 3 * tokens(1, N, 96, 0, BF, g)
        check_backward(dy, x, w, rpb.linear_backward(dy, x, w, input_pre=ipre, input_activation=act), ipre, act)


@pytest.mark.parametrize("act", ACTS[2:])
@pytest.mark.parametrize("B,N,K,out,d,dt", [(1, 2500, 200, 2056, 0, BF), (3, 700, 384, 2088, 64, HF), (1, 5001, 768, 2128, 0, HF),
                                            (2, 4900, 1024, 1024, 64, BF)])
def test_long_epilogues(act, B, N, K, out, d, dt):
    """Short contractions of many tiles, whose epilogue takes longer than their products."""
    g = torch.Generator().manual_seed(12)
    x = tokens(B, N, K, d, dt, g)
    w = (torch.randn(out, K, generator=g) * K ** -0.5).to(dt).cuda()
    b = torch.randn(out, generator=g).cuda()
    y, pre = rpb.linear(x, w, b, activation=act, keep_pre=True)
    check_forward(x, w, y, b, act, None, pre)
    assert torch.equal(rpb.linear(x, w, b, activation=act), y)
    dy = torch.randn(B, N, K, generator=g).to(dt).cuda()            # and back through a layer after it
    ipre = tokens(B, N, out // 64 * 64, d, dt, g)
    wb = (torch.randn(K, out // 64 * 64, generator=g) * K ** -0.5).to(dt).cuda()
    for gd in (dt, F32):
        got = rpb.linear_backward(dy, ipre, wb, input_pre=ipre, input_activation=act, weight_grad=False, bias_grad=False, grad_dtype=gd)
        check_backward(dy, ipre, wb, got, ipre, act)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("n", [1, 8, 1000, 1003, 40960])
@pytest.mark.parametrize("dt,zd,od", [(BF, BF, BF), (HF, HF, F32), (F32, F32, F32), (BF, F32, BF)])
def test_activation_backward(act, n, dt, zd, od):
    g = torch.Generator().manual_seed(3)
    pre, dy = (4 * torch.randn(n, generator=g)).to(dt).cuda(), torch.randn(n, generator=g).to(zd).cuda()
    got = rpb.activation_backward(dy, pre, act, grad_dtype=od)
    p64, d64 = f64(pre), f64(dy)
    want = d64 * ob.activation_slope(p64, act)
    near(got, want, rounding(want, od) + np.abs(d64) * tol.slope(p64, act), act)


def test_activation_values_far_out():
    """Every activation and slope is what it tends to, and NaN stays."""
    inf = float("inf")
    pre = torch.tensor([inf, 1e30, 100.0, 0.0, -100.0, -1e30, -inf, float("nan")], device="cuda")
    one = torch.ones(8, device="cuda")
    for act in ACTS[1:]:
        s = rpb.activation_backward(one, pre, act).tolist()
        assert s[0] == s[1] == s[2] == 1.0, (act, s)
        assert all(abs(v) < 1e-20 for v in s[4:7]), (act, s)
        if act != "relu":
            # gelu's fit of Phi(-z) is 2^-20 relative off everywhere, at 0 too: 2^-21 of a half
            assert abs(s[3] - 0.5) <= 2.0 ** -20 and s[7] != s[7], (act, s)


@pytest.mark.parametrize("act", ACTS[1:])
def test_a_nan_stays_alone(act):
    """Neighbours share instructions, and gelu's a reciprocal (of the product of two arguments, so that last bits depend on the
    neighbour): none of a NaN or an infinity."""
    g = torch.Generator().manual_seed(11)
    pre = torch.randn(64, generator=g).cuda()
    one = torch.ones(64, device="cuda")
    for k, bad in ((5, float("nan")), (8, float("inf")), (11, -float("inf")), (14, 3e38)):
        pre[k] = bad
    got = rpb.activation_backward(one, pre, act)
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[[5, 8, 11, 14]] = False
    u = pre[keep].double().cpu().numpy()
    near(got[keep], ob.activation_slope(u, act), tol.slope(u, act) + 2.0 ** -24, act)
    for N in (7, 200):   # and in the forward: a bias of such values makes whole columns of them
        x = torch.zeros(N, 64, device="cuda", dtype=BF)
        y = rpb.linear(x, torch.zeros(64, 64, device="cuda", dtype=BF), pre, activation=act, out_dtype=F32)
        want = ob.activation(u, act)
        near(y[:, keep], np.broadcast_to(want, (N, len(want))), rounding(want, F32) + tol.act(u, act), act)
        assert y[:, 5].isnan().all()


@pytest.mark.parametrize("N", [9, 200])
def test_strides(N):
    """Slices of a packed buffer, batches and heads in any order, for input and gradient."""
    g = torch.Generator().manual_seed(4)
    packed = torch.randn(2, N, 5, 128, generator=g).to(BF).cuda()
    w = (torch.randn(72, 128, generator=g) / 11).to(BF).cuda()
    for x in (packed[:, :, 1], packed[:, :, 3].transpose(0, 1)):
        check_forward(x, w, rpb.linear(x, w))
        dy = torch.randn(x.shape[0], x.shape[1], 72, generator=g).to(BF).cuda()
        check_backward(dy, x, w, rpb.linear_backward(dy, x, w))
    wh = (torch.randn(72, 384, generator=g) / 20).to(BF).cuda()
    x = packed[:, :, 1:4]                      # heads side by side in wider rows
    check_forward(x, wh, rpb.linear(x, wh))
    x = packed[:, :, 0:5:2]                    # every other head
    check_forward(x, wh, rpb.linear(x, wh))
    dy = torch.randn(2, N, 72, generator=g).to(BF).cuda()
    check_backward(dy, x, wh, rpb.linear_backward(dy, x, wh))
    # two dimensions and one
    x2 = packed[0, :, 2]
    assert torch.equal(rpb.linear(x2, w), rpb.linear(x2.contiguous()[None], w)[0])
    assert torch.equal(rpb.linear(x2[3], w), rpb.linear(x2[3:4], w)[0])


def test_some_gradients():
    g = torch.Generator().manual_seed(5)
    x, w = tokens(2, 50, 64, 0, HF, g), torch.randn(72, 64, generator=g).to(HF).cuda()
    dy = torch.randn(2, 50, 72, generator=g).to(HF).cuda()
    full = rpb.linear_backward(dy, x, w)
    for keep in range(8):
        flags = [bool(keep >> i & 1) for i in range(3)]
        got = rpb.linear_backward(dy, x, w, input_grad=flags[0], weight_grad=flags[1], bias_grad=flags[2])
        for f, p, q in zip(flags, got, full):
            assert p is None if not f else torch.equal(p, q)


@pytest.mark.parametrize("N", [3, 140])
def test_rows_past_an_edge_do_not_matter(N):
    """Infinities right behind a strided input's rows and features stay out."""
    g = torch.Generator().manual_seed(6)
    buf = torch.full((2, N + 9, 200), float("inf"), dtype=BF, device="cuda")
    x = buf[:, :N, :72]
    x.copy_(torch.randn(2, N, 72, generator=g))
    w = torch.randn(40, 72, generator=g).to(BF).cuda()
    dy = torch.randn(2, N, 40, generator=g).to(BF).cuda()
    check_forward(x, w, rpb.linear(x, w))
    check_backward(dy, x, w, rpb.linear_backward(dy, x, w))


def test_no_tokens():
    x, w = torch.zeros(3, 0, 64, device="cuda", dtype=BF), torch.ones(72, 64, device="cuda", dtype=BF)
    assert rpb.linear(x, w).shape == (3, 0, 72)
    dx, dw, db = rpb.linear_backward(torch.zeros(3, 0, 72, device="cuda", dtype=BF), x, w)
    assert dx.shape == x.shape and not dw.any() and not db.any()
    e = torch.zeros(0, device="cuda", dtype=BF)
    assert rpb.activation_backward(e, e, "gelu").shape == (0,)


@pytest.mark.parametrize("N", [4, 700])
def test_streams_and_graphs(N):
    g = torch.Generator().manual_seed(7)
    x, w = tokens(2, N, 192, 64, BF, g), torch.randn(264, 192, generator=g).to(BF).cuda()
    b = torch.randn(264, generator=g).to(BF).cuda()
    dy = torch.randn(2, N, 264, generator=g).to(BF).cuda()

    def step(stream=None):
        return (rpb.linear(x, w, b, activation="silu", stream=stream), *rpb.linear_backward(dy, x, w, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step())
        graphs.append(gr)
    s2 = torch.cuda.Stream()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(want, o))
    assert rpb.device_status() == 0


@pytest.mark.parametrize("N", [5, 140, 1000])
@pytest.mark.parametrize("gd", [BF, F32])
@pytest.mark.parametrize("heads,d", [(1, 136), (3, 64)])
def test_a_gradient_into_a_larger_buffer(N, gd, heads, d):
    """dx by strides of the caller's: the rows, heads and columns beside it are left as they were."""
    B, K, out = 2, heads * d, 264
    g = torch.Generator().manual_seed(15)
    x = tokens(B, N, K, 0, BF, g)
    w, dy = torch.randn(out, K, generator=g).to(BF).cuda(), torch.randn(B, N, out, generator=g).to(BF).cuda()
    want = rpb.linear_backward(dy, x, w, weight_grad=False, bias_grad=False, grad_dtype=gd)[0]
    buf = torch.full((B, N + 3, heads + 1, d + 16), 7.0, dtype=gd, device="cuda")
    sb, sn, sh, _ = buf.stride()
    at = torch.tensor([buf.data_ptr(), sb, sn, sh], dtype=torch.int64).numpy().tobytes()
    code = {BF: rpb.DERA_BF16, F32: rpb.DERA_F32}[gd]
    assert rpb.load_library().dera_linear_backward(dy.data_ptr(), None, w.data_ptr(), None, at, None, None, B, N, heads, d, out, 0,
                                                   rpb.DERA_BF16, code, rpb.DERA_F32, None, 0,
                                                   torch.cuda.current_stream().cuda_stream) == 0
    got = buf[:, :N, :heads, :d].reshape(B, N, K)
    # tiles may lie otherwise, and sums be taken in another order
    near(got, f64(want), 2 * rounding(f64(want), gd) + 2 * tol.product(flat(dy, out), f64(w).T).reshape(B, N, K), "dx")
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[:, :N, :heads, :d] = False
    assert (buf[keep] == 7.0).all()


def test_workspaces():
    """A caller's own, of exactly the size, with anything in it; too small, off its alignment and none at all are refused."""
    g = torch.Generator().manual_seed(12)
    x, w = tokens(2, 3000, 128, 64, BF, g), torch.randn(264, 128, generator=g).to(BF).cuda()
    dy = torch.randn(2, 3000, 264, generator=g).to(BF).cuda()
    need = rpb.linear_backward_workspace_size(2, 3000, 2, 64, 264)
    ws = torch.full((need + 16,), 0xff, dtype=torch.uint8, device="cuda")
    want = rpb.linear_backward(dy, x, w)
    got = rpb.linear_backward(dy, x, w, workspace=ws[:need])
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and (ws[need:] == 0xff).all()
    for bad, status in ((ws[:need - 1], 9), (ws[16:], 5)):
        with pytest.raises(rpb.DeraError) as e:
            rpb.linear_backward(dy, x, w, workspace=bad)
        assert e.value.status == status
    assert torch.equal(rpb.linear_backward(dy, x, w, weight_grad=False, bias_grad=False, workspace=ws[:1])[0], want[0])


def test_two_streams_at_once():
    """Calls on two streams that overlap, and a third that reads what the first wrote."""
    g = torch.Generator().manual_seed(13)
    x, w = tokens(1, 4000, 256, 0, BF, g), torch.randn(1032, 256, generator=g).to(BF).cuda()
    dy = torch.randn(1, 4000, 1032, generator=g).to(BF).cuda()
    want = (rpb.linear(x, w, activation="gelu"), *rpb.linear_backward(dy, x, w))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            outs.append((rpb.linear(x, w, activation="gelu", stream=s), *rpb.linear_backward(dy, x, w, stream=s)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(want, o))


def test_fp32_results_are_summed_finely():
    """y, dx and dW in fp32 over long contractions, with few tokens and many: of one size, so that cutting towards zero would add up."""
    g = torch.Generator().manual_seed(14)
    for N in (9, 300, 3000):
        x = (1 + 0.1 * torch.rand(1, N, 4096, generator=g)).to(BF).cuda()
        w = (1 + 0.1 * torch.rand(264, 4096, generator=g)).to(BF).cuda()
        dy = (1 + 0.1 * torch.rand(1, N, 264, generator=g)).to(BF).cuda()
        y, (dx, dw, _) = rpb.linear(x, w, out_dtype=F32)[0], rpb.linear_backward(dy, x, w)
        x64, w64, d64 = x[0].double(), w.double(), dy[0].double()
        for got, want in ((y, x64 @ w64.T), (dx[0], d64 @ w64), (dw, d64.T @ x64)):
            # 32 cuts of a chain, at most 2^-22 each, and as many roundings of 2^-24 for the chains
            assert float(((got.double() - want) / want).abs().max()) <= 32 * 2.0 ** -22 + 64 * 2.0 ** -24


def test_many_tokens_sum_as_finely():
    """dweight in fp32 over more tokens than one chain of the tensor core's sums takes: of ones, every bit."""
    for N in (4096, 20000):
        x = torch.ones(N, 64, device="cuda", dtype=BF)
        dw = rpb.linear_backward(torch.ones(N, 72, device="cuda", dtype=BF), x, torch.ones(72, 64, device="cuda", dtype=BF),
                                 input_grad=False)[1]
        assert torch.equal(dw, torch.full((72, 64), float(N), device="cuda"))
    g = torch.Generator().manual_seed(8)
    x, dy = torch.randn(30000, 64, generator=g).to(BF).cuda(), torch.randn(30000, 64, generator=g).to(BF).cuda()
    dw = rpb.linear_backward(dy, x, x[:64], input_grad=False)[1]
    want = dy.double().T @ x.double()
    assert float((dw.double() - want).norm() / want.norm()) < 1e-5


def test_offsets_past_two_to_the_31():
    N, K = (1 << 31) // 4096 + 200, 4096
    x = torch.zeros(N, K, device="cuda", dtype=BF)
    tail = torch.randn(140, K, device="cuda").to(BF)
    x[-140:] = tail
    w = (torch.randn(4096, K, device="cuda") / 64).to(BF)
    y = rpb.linear(x, w)
    assert torch.allclose(y[-140:].float(), rpb.linear(tail, w).float(), rtol=2 ** -7, atol=1e-2)
    assert not y[:-140].any()
    dx, dw, db = rpb.linear_backward(y, x, w, grad_dtype=BF)
    dx2, dw2, db2 = rpb.linear_backward(y[-140:].contiguous(), tail, w, grad_dtype=BF)
    assert torch.allclose(dx[-140:].float(), dx2.float(), rtol=2 ** -7, atol=1e-2) and not dx[:-140].any()
    assert torch.allclose(dw, dw2, rtol=1e-4, atol=1e-3) and torch.allclose(db, db2, rtol=1e-4, atol=1e-3)


@pytest.mark.parametrize("N,K,out", [(20, 512, 768), (196, 768, 768), (1369, 768, 1000), (4900, 1024, 512)])
def test_gradients_end_before_what_follows(N, K, out):
    """The kernels of a backward run into one another: what is enqueued after the call may overwrite all that it read, and read all that
    it wrote, with or without each gradient."""
    g = torch.Generator().manual_seed(13)
    dy0, x0 = torch.randn(N, out, generator=g).to(BF).cuda(), torch.randn(N, K, generator=g).to(BF).cuda()
    w0 = (torch.randn(out, K, generator=g) / 30).to(BF).cuda()
    ws = torch.empty(rpb.linear_backward_workspace_size(1, N, 1, K, out), dtype=torch.uint8, device="cuda")
    which = [dict(input_grad=i, weight_grad=j, bias_grad=k) for i in (True, False) for j in (True, False) for k in (True, False) if i or j or k]
    want = []
    for kw in which:
        want.append(rpb.linear_backward(dy0, x0, w0, **kw))
        torch.cuda.synchronize()
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    dy, x, w = dy0.clone(), x0.clone(), w0.clone()
    for _ in range(30):
        for kw, ref in zip(which, want):
            got = rpb.linear_backward(dy, x, w, workspace=ws, **kw)
            for t in (dy, x, w):
                t.fill_(float("nan"))
            ws.fill_(255)
            for a, b in zip(got, ref):
                if a is not None:
                    bad += (a != b).sum()
            for t, t0 in ((dy, dy0), (x, x0), (w, w0)):
                t.copy_(t0)
    assert bad.item() == 0
