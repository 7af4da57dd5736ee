"""qk_norm_rope and its backward against the CPU float64 oracle.

Tolerances, derived from the arithmetic: everything is fp32 and rounded once, so an output may be
off by half a step of its type (eps / 2 relative; fp16 subnormals by 2^-25), plus the fp32
errors of about a dozen operations on terms of the row's size: 2^-19 of the largest term
(16 roundings of 2^-24 and the 2^-22 of the reciprocal square root come to less).  A weight's gradient is a sum
over all rows in fp32: 2^-18 of the sum of the terms' sizes covers chains of up to 64 additions,
which no case here passes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(B, N, hq, hk, d, dtype, norm, rot, inter, table, seed=0, wdtype=None):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, N, hq + 2 * hk, d, generator=g) * torch.exp(0.5 * torch.randn(hq + 2 * hk, d, generator=g))
    qkv = qkv.to(dtype).cuda()
    kw = dict(interleaved=inter)
    if norm:
        kw["q_weight"] = (1 + 0.3 * torch.randn(d, generator=g)).to(wdtype or dtype).cuda()
        kw["k_weight"] = (1 + 0.3 * torch.randn(d, generator=g)).to(wdtype or dtype).cuda()
    if rot:
        ang = 3 * torch.randn(table or N, rot // 2, generator=g)
        kw["cos"], kw["sin"] = ang.cos().cuda(), ang.sin().cuda()
        if table:
            kw["positions"] = torch.randint(0, table, (B, N), generator=g).int().cuda()
    dz = [torch.randn(B * h, N, d, generator=g).to(dtype).cuda() for h in (hq, hk, hk)]
    return qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:], kw, dz


def near(got, want, size, dtype, what):
    """got within half a step of want, plus 2^-19 of `size` (broadcast against want)."""
    g = f64(got)
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0 ** -19 * size + (2.0 ** -25 if dtype == HF else 0)
    assert g.shape == want.shape and np.isfinite(g).all(), what
    worst = (np.abs(g - want) - tol).max()
    assert worst <= 0, f"{what}: {worst:.3e} over its tolerance"


CASES = {
    # B, N, q heads, kv heads, d, dtype, norm, rotary_dim, interleaved, table rows (0: no positions)
    "token": (5, 1, 4, 2, 128, BF, True, 128, False, 33),
    "one": (1, 1, 1, 1, 64, HF, True, 64, True, 1),
    "grid": (1, 100, 3, 3, 64, BF, True, 64, False, 0),
    "odd": (3, 37, 5, 1, 64, HF, True, 32, True, 50),
    "third": (2, 33, 2, 2, 128, HF, True, 48, False, 40),
    "sixteen": (2, 17, 9, 3, 128, BF, True, 16, False, 0),
    "norm_only": (2, 21, 2, 4, 64, BF, True, 0, False, 0),
    "turn_only": (2, 21, 2, 1, 128, HF, False, 128, True, 0),
    "move_only": (2, 5, 3, 1, 64, BF, False, 0, False, 0),
    "many_heads": (2, 9, 33, 17, 64, BF, True, 64, False, 11),
    "tokens": (1, 300, 1, 1, 64, BF, True, 64, False, 0),
}


def oracle_kw(kw, which):
    return dict(weight=f64(kw.get(f"{which}_weight")), cos=f64(kw.get("cos")), sin=f64(kw.get("sin")),
                positions=None if kw.get("positions") is None else kw["positions"].cpu().numpy(),
                interleaved=kw["interleaved"])


def check_forward(q, k, v, kw, outs, dtype, what):
    for name, x, out in (("q", q, outs[0]), ("k", k, outs[1])):
        want = oracle.qk_norm_rope(f64(x), **oracle_kw(kw, name))
        near(out, want, np.abs(want).max(-1, keepdims=True), dtype, f"{what} {name}")
    if v is not None:
        B, N, h, d = v.shape
        assert torch.equal(outs[2], v.transpose(1, 2).reshape(B * h, N, d))


def check_backward(q, k, kw, dz, grads, dtype, what):
    for i, (name, x) in enumerate((("q", q), ("k", k))):
        okw = oracle_kw(kw, name)
        dx, dw = oracle.qk_norm_rope_backward(f64(x), f64(dz[i]), **okw)
        xf = f64(x)
        size = np.abs(f64(dz[i])).reshape(x.shape[0], x.shape[2], x.shape[1], -1).transpose(0, 2, 1, 3).max(-1, keepdims=True) * 2
        if dw is not None:
            r = 1 / np.sqrt((xf * xf).mean(-1, keepdims=True) + 1e-6)
            wmax = np.abs(okw["weight"]).max()
            size = size * wmax * r * (1 + np.abs(xf * r).max(-1, keepdims=True) ** 2)
        near(grads[i], dx, size, dtype, f"{what} d{name}")
        if dw is None:
            assert grads[3 + i] is None
            continue
        back, _ = oracle.qk_norm_rope_backward(f64(x), f64(dz[i]), **{**okw, "weight": None})
        terms = np.abs(back * xf * r).sum((0, 1, 2))
        got = f64(grads[3 + i])
        assert (np.abs(got - dw) <= 2.0 ** -18 * terms).all(), f"{what} d{name}_weight"


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name):
    q, k, v, kw, _ = make(*CASES[name])
    outs = rpb.qk_norm_rope(q, k, v, **kw)
    check_forward(q, k, v, kw, outs, CASES[name][5], name)
    two = rpb.qk_norm_rope(q, k, **kw)
    assert len(two) == 2 and torch.equal(two[0], outs[0]) and torch.equal(two[1], outs[1])


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("name", sorted(CASES))
def test_backward(name, fp32):
    dtype = CASES[name][5]
    q, k, v, kw, dz = make(*CASES[name], seed=1, wdtype=torch.float32 if fp32 else None)
    if fp32:
        dz = [t.float() * 1.2345 for t in dz]
    gd = torch.float32 if fp32 else dtype
    grads = rpb.qk_norm_rope_backward(q, k, *dz, grad_dtype=gd, **kw)
    check_backward(q, k, kw, dz, grads, gd, name)
    want = f64(dz[2]).reshape(k.shape[0], k.shape[2], k.shape[1], -1).transpose(0, 2, 1, 3)
    near(grads[2], want, 0.0, gd, f"{name} dv")
    again = rpb.qk_norm_rope_backward(q, k, *dz, grad_dtype=gd, **kw)
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b)


def test_tiny_and_huge_rows():
    """Rows of zeros, of the smallest and of large values: the norm stays finite, its gradient too."""
    q, k, v, kw, dz = make(1, 6, 2, 2, 64, BF, True, 64, False, 0)
    q = q.clone()
    q[0, 0] = 0
    q[0, 1] = 1e-30
    q[0, 2] = 3e18      # its square still fits fp32
    q[0, 3, :, 1:] = 0  # one element alone
    outs = rpb.qk_norm_rope(q, k, v, **kw)
    check_forward(q, k, v, kw, outs, BF, "rows")
    assert torch.count_nonzero(outs[0].view(1, 2, 6, 64)[:, :, 0]) == 0
    grads = rpb.qk_norm_rope_backward(q, k, *dz, **kw)
    check_backward(q, k, kw, dz, grads, torch.float32, "rows")


def test_strides_and_packed_gradient():
    """Inputs in another order of dimensions, repeated rows, and gradients written into the slices of
    one packed buffer whose other rows stay as they were."""
    B, N, hq, hk, d = 2, 19, 4, 2, 64
    q, k, v, kw, dz = make(B, N, hq, hk, d, BF, True, 64, False, 0, seed=3)
    want = rpb.qk_norm_rope(q, k, v, **kw)
    byhead = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)     # [heads][B][N][d] in memory
    got = rpb.qk_norm_rope(byhead, k, v, **kw)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    one = k[:, :, :1].expand(B, N, 3, d)                                # stride 0 over heads
    rep = rpb.qk_norm_rope(q, one, one, **kw)
    ref = rpb.qk_norm_rope(q, one.contiguous(), one.contiguous(), **kw)
    for a, b in zip(rep, ref):
        assert torch.equal(a, b)
    ref = rpb.qk_norm_rope_backward(q, k, *dz, grad_dtype=BF, **kw)
    packed = torch.full((B, N + 2, hq + 2 * hk + 1, d), 7.0, dtype=BF, device="cuda")
    view = packed[:, 1:N + 1]
    out = rpb.qk_norm_rope_backward(q, k, *dz, dq=view[:, :, :hq], dk=view[:, :, hq:hq + hk],
                                    dv=view[:, :, hq + hk:hq + 2 * hk], **kw)
    for a, b in zip(out, ref):
        assert torch.equal(a, b)
    assert (packed[:, 0] == 7).all() and (packed[:, -1] == 7).all() and (packed[:, :, -1] == 7).all()


def test_position_outside_the_table_is_nan():
    q, k, v, kw, dz = make(2, 5, 2, 1, 64, BF, True, 32, False, 9, seed=4)
    want = rpb.qk_norm_rope(q, k, v, **kw)
    kw["positions"] = kw["positions"].clone()
    kw["positions"][0, 1], kw["positions"][1, 4] = 9, -1
    got = rpb.qk_norm_rope(q, k, v, **kw)
    for a, w, h in zip(got[:2], want, (2, 1)):
        a, w = a.view(2, h, 5, 64), w.view(2, h, 5, 64)
        for b, n in ((0, 1), (1, 4)):
            assert a[b, :, n, :32].isnan().all() and torch.equal(a[b, :, n, 32:], w[b, :, n, 32:])
        keep = torch.ones(2, 5, dtype=torch.bool)
        keep[0, 1] = keep[1, 4] = False
        assert torch.equal(a.transpose(1, 2)[keep], w.transpose(1, 2)[keep])
    assert torch.equal(got[2], want[2])
    dq = rpb.qk_norm_rope_backward(q, k, *dz, **kw)[0]
    assert dq[0, 1].isnan().all() and dq[1, 4].isnan().all() and not dq[0, 0].isnan().any()


def test_empty():
    for shape in ((0, 4, 2, 64), (3, 0, 2, 64)):
        e = torch.empty(shape, dtype=BF, device="cuda")
        w = torch.ones(64, dtype=BF, device="cuda")
        out = rpb.qk_norm_rope(e, e, e, q_weight=w, k_weight=w)
        assert out[0].shape == (shape[0] * 2, shape[1], 64)
        z = torch.empty((shape[0] * 2, shape[1], 64), dtype=BF, device="cuda")
        grads = rpb.qk_norm_rope_backward(e, e, z, z, z, q_weight=w, k_weight=w)
        assert grads[0].shape == shape
        assert torch.count_nonzero(grads[3]) == 0 and torch.count_nonzero(grads[4]) == 0


def test_graph_and_other_stream():
    """Captured once and replayed on new inputs; on a stream other than the current one."""
    q, k, v, kw, dz = make(2, 50, 3, 3, 64, BF, True, 64, False, 60, seed=5)
    ws = torch.empty(rpb.qk_norm_rope_backward_workspace_size(2, 50, 3, 3, 64), dtype=torch.uint8, device="cuda")

    def both(**more):
        return (*rpb.qk_norm_rope(q, k, v, **kw, **more), *rpb.qk_norm_rope_backward(q, k, *dz, **kw, workspace=ws, **more))

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for t in (q, k, v, *dz):
        t.mul_(-0.5)
    graph.replay()
    want = both()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_largest_head_count_and_long_rows():
    """Heads up to the limit in one dimension of the grid, and a token axis past a block's runs."""
    q, k, v, kw, dz = make(1, 2, 16384, 1, 64, BF, True, 64, False, 0, seed=7)
    check_forward(q, k, v, kw, rpb.qk_norm_rope(q, k, v, **kw), BF, "heads")
    q, k, v, kw, dz = make(3, 9001, 1, 1, 64, HF, True, 64, True, 0, seed=8)
    check_forward(q, k, v, kw, rpb.qk_norm_rope(q, k, v, **kw), HF, "tokens")
    grads = rpb.qk_norm_rope_backward(q, k, *dz, grad_dtype=HF, **kw)
    for i, (name, x) in enumerate((("q", q), ("k", k))):
        okw = oracle_kw(kw, name)
        _, dw = oracle.qk_norm_rope_backward(f64(x), f64(dz[i]), **okw)
        back, _ = oracle.qk_norm_rope_backward(f64(x), f64(dz[i]), **{**okw, "weight": None})
        xf = f64(x)
        terms = np.abs(back * xf / np.sqrt((xf * xf).mean(-1, keepdims=True) + 1e-6)).sum((0, 1, 2))
        assert (np.abs(f64(grads[3 + i]) - dw) <= 2.0 ** -18 * terms).all()


def test_other_device_tensors_are_refused():
    q, k, v, kw, dz = make(1, 4, 2, 1, 64, BF, True, 64, False, 0)
    kw["cos"] = kw["cos"].cpu()
    with pytest.raises(rpb.DeraError) as e:
        rpb.qk_norm_rope(q, k, v, **kw)
    assert e.value.status == 6


def test_offsets_past_32_bits():
    """A packed projection of more than 2^31 elements, forward and backward: the last batch is what a call on it
    alone gives, bit for bit (rows are independent of one another)."""
    if torch.cuda.mem_get_info()[0] < 80e9:
        pytest.skip("needs 80 GB")
    B, N, h, d = 240, 4096, 12, 64
    g = torch.Generator(device="cuda").manual_seed(19)
    x = torch.empty(B, N, 3 * h, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    assert x.numel() > 2 ** 31
    w = torch.rand(d, generator=g, device="cuda") + 0.5
    cos, sin = (torch.rand(N, d // 2, generator=g, device="cuda") for _ in range(2))
    kw = dict(q_weight=w, k_weight=w, cos=cos, sin=sin)

    def heads(t):
        return t[:, :, :h], t[:, :, h:2 * h], t[:, :, 2 * h:]
    z = rpb.qk_norm_rope(*heads(x), **kw)
    one = x[-1:].clone()
    z1 = rpb.qk_norm_rope(*heads(one), **kw)
    assert all(torch.equal(a[-h:], b) for a, b in zip(z, z1))
    dx = torch.empty_like(x)
    rpb.qk_norm_rope_backward(*heads(x)[:2], *z, **kw, **dict(zip(("dq", "dk", "dv"), heads(dx))))
    d1 = rpb.qk_norm_rope_backward(*heads(one)[:2], *z1, **kw, grad_dtype=torch.bfloat16)
    assert all(torch.equal(a[-1:], b) for a, b in zip(heads(dx), d1))
