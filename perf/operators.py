"""The training operators around the attention, as they are measured.

Five kinds of case, each one pass of an operator:

  qkv       qk_norm_rope: the packed projection's heads normed, rotated and laid out for the attention
  qkv_grad  qk_norm_rope_backward
  attn      attention_lse: the compact-bias attention with its log-sum-exp
  attn_grad attention_backward: dq, dk, dv and the gradients of the compact bias
  tables    project_backward: the tables' gradients and dq's part through the projection

``own`` selects between the plain form (elementary torch operations in 32 bits) and the library's
entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LOG2E = 1.4426950408889634
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def listed() -> list[dict]:
    return [
        # one new token in each of 32 sequences: grouped heads, positions looked up, latency counts
        dict(name="qkv_token", op="qkv", B=32, N=1, Hq=16, Hk=4, d=128, dtype="bf16", norm=True, rot=128,
             interleaved=False, table=4096),
        # a batch of wide 64x64 encoders with head_dim 128, half of each head rotated: bandwidth
        dict(name="qkv_wide64", op="qkv", B=8, N=4096, Hq=16, Hk=16, d=128, dtype="f16", norm=True, rot=64,
             interleaved=True, table=0),
        # the windowed blocks of one image: 25 windows of 14x14 tokens
        dict(name="qkv_grad_window14", op="qkv_grad", B=25, N=196, Hq=12, Hk=12, d=64, dtype="bf16", norm=True, rot=64,
             interleaved=False, table=0),
        # eight 64x64 encoders in one training step
        dict(name="qkv_grad_batched64", op="qkv_grad", B=8, N=4096, Hq=12, Hk=12, d=64, dtype="bf16", norm=True, rot=64,
             interleaved=False, table=0),
        # the windows of one image with a 16-bit bias whose padded rows and columns are masked
        dict(name="attn_window14", op="attn", BH=300, H=14, W=14, d=64, dtype="bf16", bias="bf16", mask="edge"),
        # the batched wide encoder, global attention
        dict(name="attn_wide64", op="attn", BH=64, H=64, W=64, d=64, dtype="bf16", bias="f32", mask="none"),
        # the smallest training call: two heads of a 16x16 grid
        dict(name="attn_grad_grid16", op="attn_grad", BH=2, H=16, W=16, d=64, dtype="bf16", bias="f32", mask="none"),
        # one image's global attention
        dict(name="attn_grad_global64", op="attn_grad", BH=12, H=64, W=64, d=64, dtype="bf16", bias="f32", mask="none"),
        # 16 images of different sizes padded to 40x40: rows that the mask leaves empty
        dict(name="attn_grad_ragged40", op="attn_grad", BH=192, H=40, W=40, d=64, dtype="f16", bias="f32", mask="empty"),
        # one image with head_dim 128
        dict(name="attn_grad_global64d128", op="attn_grad", BH=12, H=64, W=64, d=128, dtype="bf16", bias="f32",
             mask="none"),
        # the windows' tables
        dict(name="tables_window14", op="tables", BH=300, H=14, W=14, d=64, dtype="bf16", dq="bf16"),
        # eight images' tables
        dict(name="tables_batched64", op="tables", BH=96, H=64, W=64, d=64, dtype="bf16", dq="bf16"),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng) -> dict:
    op = rng.choice(["qkv", "qkv_grad", "attn", "attn_grad", "attn_grad", "tables"])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("qkv", "qkv_grad"):
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        N = _log_int(rng, 1, 5000)
        # tokens x heads x d of the larger listed case of the kind
        most = (8 * 4096 * 48 * 128 if op == "qkv" else 8 * 4096 * 36 * 64) // ((Hq + 2 * Hk) * d * N)
        if most < 1:
            N, most = 512, max(1, (8 * 4096 * 36 * 64) // ((Hq + 2 * Hk) * d * 512))
        B = _log_int(rng, 1, min(most, 300))
        rot = rng.choice([0, 16, 48, d // 2, d, d])
        norm = rot == 0 or rng.random() < 0.8
        return dict(op=op, B=B, N=N, Hq=Hq, Hk=Hk, d=d, dtype=dtype, norm=norm, rot=rot,
                    interleaved=rng.random() < 0.4, table=rng.choice([0, N + 7, 9000]) if rot else 0)
    H, W = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
    N = H * W
    if op == "tables":
        BH = _log_int(rng, 1, max(1, min(400, (96 * 4096 * 128 * 64) // (N * (H + W) * d))))
        return dict(op=op, BH=BH, H=H, W=W, d=d, dtype=dtype, dq=rng.choice(["none", "f32", dtype]))
    most = (64 if op == "attn" else 12) * 4096 * 4096 * 64 // (N * N * d)
    BH = _log_int(rng, 1, max(1, min(400, most)))
    return dict(op=op, BH=BH, H=H, W=W, d=d, dtype=dtype, bias=rng.choice(["f32", "f32", "bf16", "f16"]),
                mask=rng.choice(["none", "edge", "empty"]))


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed: int) -> torch.Generator:
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, s: float = 1.0, dtype=torch.float32) -> torch.Tensor:
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


def _prepare_qkv(case: dict, seed: int) -> dict:
    g, t = _gen(seed), DTYPES[case["dtype"]]
    B, N, Hq, Hk, d, rot = (case[k] for k in ("B", "N", "Hq", "Hk", "d", "rot"))
    # channels of unequal size, as a projection gives them
    chan = 0.5 + 1.5 * torch.rand(Hq + 2 * Hk, d, generator=g, device="cuda")
    qkv = torch.randn(B, N, Hq + 2 * Hk, d, generator=g, device="cuda", dtype=t).mul_(chan.to(t))
    s = dict(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hk], v=qkv[:, :, Hq + Hk:], interleaved=case["interleaved"])
    s["qw"] = _randn(g, d, s=0.2).add_(1).to(t) if case["norm"] else None
    s["kw"] = _randn(g, d, s=0.2).add_(1).to(t) if case["norm"] else None
    s["cos"] = s["sin"] = s["pos"] = None
    if rot:
        rows = case["table"] or N
        freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
        ang = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        if case["table"]:
            s["pos"] = torch.randint(0, rows, (B, N), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "qkv_grad":
        s["dq"] = torch.randn(B * Hq, N, d, generator=g, device="cuda", dtype=t)
        s["dk"] = torch.randn(B * Hk, N, d, generator=g, device="cuda", dtype=t)
        s["dv"] = torch.randn(B * Hk, N, d, generator=g, device="cuda", dtype=t)
    return s


def _mask_bias(case: dict, g, rel_h: torch.Tensor, rel_w: torch.Tensor) -> None:
    """Every problem its own valid area; "edge" masks the keys outside it with the type's lowest
    value, "empty" with -inf, and for the queries outside it every key."""
    BH, H, W = case["BH"], case["H"], case["W"]
    vh = torch.randint((H + 1) // 2, H + 1, (BH, 1, 1), generator=g, device="cuda")
    vw = torch.randint((W + 1) // 2, W + 1, (BH, 1, 1), generator=g, device="cuda")
    low = torch.finfo(rel_h.dtype).min if case["mask"] == "edge" else -math.inf
    rel_h.masked_fill_(torch.arange(H, device="cuda") >= vh, low)
    rel_w.masked_fill_(torch.arange(W, device="cuda") >= vw, low)
    if case["mask"] == "empty":
        n = torch.arange(H * W, device="cuda").view(1, -1, 1)
        rel_h.masked_fill_((n // W >= vh) | (n % W >= vw), -math.inf)


def _prepare_attn(case: dict, seed: int) -> dict:
    g, t = _gen(seed), DTYPES[case["dtype"]]
    BH, H, W, d = (case[k] for k in ("BH", "H", "W", "d"))
    N = H * W
    s = dict(H=H, W=W, scale=d ** -0.5)
    for name in ("q", "k", "v"):
        s[name] = _randn(g, BH, N, d, dtype=t)
    # the size that the projection of unit queries on tables of 0.25 gives
    s["rel_h"] = _randn(g, BH, N, H, s=0.25 * math.sqrt(d), dtype=DTYPES[case["bias"]])
    s["rel_w"] = _randn(g, BH, N, W, s=0.25 * math.sqrt(d), dtype=DTYPES[case["bias"]])
    if case["mask"] != "none":
        _mask_bias(case, g, s["rel_h"], s["rel_w"])
    if case["op"] == "attn_grad":
        # what the forward pass of the step left behind
        out = torch.empty(BH, N, d, device="cuda", dtype=t)
        lse = torch.empty(BH, N, device="cuda")
        step = max(1, (1 << 28) // (N * N))
        for b in range(0, BH, step):
            part = slice(b, b + step)
            z = torch.baddbmm(((s["rel_h"][part].float()[..., None] + s["rel_w"][part].float()[..., None, :])
                               .flatten(2)), s["q"][part].float(), s["k"][part].float().mT, alpha=s["scale"])
            top = z.amax(-1, keepdim=True).clamp_min_(-1e37)
            z.sub_(top).exp_()
            tot = z.sum(-1, keepdim=True)
            out[part] = (z @ s["v"][part].float() / tot.where(tot > 0, 1.0)).to(t)
            lse[part] = (top * LOG2E + tot.log2()).squeeze(-1)
        s["out"], s["lse"] = out, lse
        s["dout"] = _randn(g, BH, N, d, dtype=t)
    return s


def _prepare_tables(case: dict, seed: int) -> dict:
    g, t = _gen(seed), DTYPES[case["dtype"]]
    BH, H, W, d = (case[k] for k in ("BH", "H", "W", "d"))
    N = H * W
    s = dict(H=H, W=W, q=_randn(g, BH, N, d, dtype=t), th=_randn(g, 2 * H - 1, d, s=0.25, dtype=t),
             tw=_randn(g, 2 * W - 1, d, s=0.25, dtype=t))
    # rows of very different size, as a softmax's gradient has them; each sums to zero
    size = 0.05 * torch.exp(torch.randn(BH, N, 1, generator=g, device="cuda"))
    for name, L in (("drel_h", H), ("drel_w", W)):
        x = torch.randn(BH, N, L, generator=g, device="cuda")
        s[name] = (x - x.mean(-1, keepdim=True)).mul_(size) if L > 1 else x.mul_(size)
    s["dq"] = None if case["dq"] == "none" else _randn(g, BH, N, d, s=0.1, dtype=DTYPES[case["dq"]])
    s["grad"] = t if case["dq"] == "none" else DTYPES[case["dq"]]
    return s


def prepare(case: dict, seed: int) -> dict:
    make = {"qkv": _prepare_qkv, "qkv_grad": _prepare_qkv, "attn": _prepare_attn, "attn_grad": _prepare_attn,
            "tables": _prepare_tables}[case["op"]]
    s = make(case, seed)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------------------------- plain forms
def _rotate(y: torch.Tensor, c: torch.Tensor, s: torch.Tensor, interleaved: bool) -> torch.Tensor:
    """Rotation of the first 2 c.shape[-1] elements of every row; the inverse with -s."""
    R = 2 * c.shape[-1]
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., :R // 2], y[..., R // 2:R])
    za, zb = a * c - b * s, b * c + a * s
    z = torch.stack((za, zb), -1).flatten(-2) if interleaved else torch.cat((za, zb), -1)
    return torch.cat((z, y[..., R:]), -1)


def _angles(s: dict) -> tuple[torch.Tensor, torch.Tensor]:
    """cos and sin as [B or 1, N, 1, R/2]."""
    if s["pos"] is None:
        return s["cos"][None, :s["q"].shape[1], None], s["sin"][None, :s["q"].shape[1], None]
    return s["cos"][s["pos"].long()][:, :, None], s["sin"][s["pos"].long()][:, :, None]


def _heads_first(x: torch.Tensor, dtype) -> torch.Tensor:
    B, N, h, d = x.shape
    return x.transpose(1, 2).reshape(B * h, N, d).to(dtype)


def _tokens_first(x: torch.Tensor, B: int) -> torch.Tensor:
    return x.unflatten(0, (B, -1)).transpose(1, 2)


def _plain_qkv(s: dict):
    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
        if s["cos"] is not None:
            y = _rotate(y, *_angles(s), s["interleaved"])
        return _heads_first(y, x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"]), _heads_first(s["v"], s["v"].dtype)


def _plain_qkv_grad(s: dict):
    def one(x, w, dz):
        dy = _tokens_first(dz.float(), x.shape[0])
        if s["cos"] is not None:
            c, sn = _angles(s)
            dy = _rotate(dy, c, -sn, s["interleaved"])
        if w is None:
            return dy.to(x.dtype).contiguous(), None
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
        xr = xf * r
        gy = dy * w.float()
        dx = r * (gy - xr * (gy * xr).mean(-1, keepdim=True))
        return dx.to(x.dtype), (dy * xr).sum(dim=(0, 1, 2))

    dq, dqw = one(s["q"], s["qw"], s["dq"])
    dk, dkw = one(s["k"], s["kw"], s["dk"])
    return dq, dk, _tokens_first(s["dv"], s["v"].shape[0]).contiguous(), dqw, dkw


def _logits(s: dict) -> torch.Tensor:
    bias = (s["rel_h"].float()[..., None] + s["rel_w"].float()[..., None, :]).flatten(2)
    return torch.baddbmm(bias, s["q"].float(), s["k"].float().mT, alpha=s["scale"])


def _plain_attn(s: dict):
    z = _logits(s)
    top = z.amax(-1, keepdim=True).clamp_min(-1e37)   # finite also for a row that is masked as a whole
    p = torch.exp(z.sub_(top))
    tot = p.sum(-1, keepdim=True)
    out = (p @ s["v"].float()) / tot.where(tot > 0, 1.0)
    return out.to(s["q"].dtype), (top * LOG2E + tot.log2()).squeeze(-1)


def _plain_attn_grad(s: dict):
    lse = s["lse"].where(s["lse"] > -math.inf, math.inf)[..., None]
    p = torch.exp2(_logits(s).mul_(LOG2E).sub_(lse))
    do, q, k, v = s["dout"].float(), s["q"].float(), s["k"].float(), s["v"].float()
    D = (do * s["out"].float()).sum(-1, keepdim=True)
    dv = p.mT @ do
    dz = p.mul_((do @ v.mT).sub_(D))
    grid = dz.unflatten(-1, (s["H"], s["W"]))
    t = s["q"].dtype
    return ((dz @ k * s["scale"]).to(t), (dz.mT @ q * s["scale"]).to(t), dv.to(t), grid.sum(-1), grid.sum(-2))


def _plain_tables(s: dict):
    H, W, q = s["H"], s["W"], s["q"].float()
    BH, d = q.shape[0], q.shape[-1]
    q = q.view(BH, H, W, d)

    def at(L):   # table row of query coordinate a and key coordinate b
        a = torch.arange(L, device=q.device)
        return a[:, None] - a[None, :] + L - 1

    def table(C, L):   # C[a, b, d] summed over a - b + L - 1 = i
        a = torch.arange(L, device=q.device)[None, :]
        b = a + L - 1 - torch.arange(2 * L - 1, device=q.device)[:, None]
        there = ((b >= 0) & (b < L))[..., None]
        return (C[a, b.clamp(0, L - 1)] * there).sum(1)

    gh, gw = s["drel_h"].view(BH, H, W, H), s["drel_w"].view(BH, H, W, W)
    dq = torch.einsum("bhwk,hkd->bhwd", gh, s["th"].float()[at(H)])
    dq = dq + torch.einsum("bhwk,wkd->bhwd", gw, s["tw"].float()[at(W)])
    dq = dq.reshape(BH, H * W, d)
    if s["dq"] is not None:
        dq = dq + s["dq"].float()
    dth = table(torch.einsum("bhwk,bhwd->hkd", gh, q), H)
    dtw = table(torch.einsum("bhwk,bhwd->wkd", gw, q), W)
    return dq.to(s["grad"]), dth, dtw


# ------------------------------------------------------------------------------------ one pass
def _own(s: dict):
    import relative_position_bias_gb300 as rpb

    if s["op"] == "qkv":
        return rpb.qk_norm_rope(s["q"], s["k"], s["v"], q_weight=s["qw"], k_weight=s["kw"], cos=s["cos"], sin=s["sin"],
                                positions=s["pos"], eps=EPS, interleaved=s["interleaved"])
    if s["op"] == "qkv_grad":
        return rpb.qk_norm_rope_backward(s["q"], s["k"], s["dq"], s["dk"], s["dv"], q_weight=s["qw"], k_weight=s["kw"],
                                         cos=s["cos"], sin=s["sin"], positions=s["pos"], eps=EPS,
                                         interleaved=s["interleaved"], grad_dtype=s["q"].dtype)
    if s["op"] == "attn":
        return rpb.attention_lse(s["q"], s["k"], s["v"], s["rel_h"], s["rel_w"], s["H"], s["W"], s["scale"])
    if s["op"] == "attn_grad":
        return rpb.attention_backward(s["q"], s["k"], s["v"], s["rel_h"], s["rel_w"], s["out"], s["lse"], s["dout"],
                                      s["H"], s["W"], s["scale"], grad_dtype=s["q"].dtype)
    return rpb.project_backward(s["q"], s["th"], s["tw"], s["drel_h"], s["drel_w"], s["H"], s["W"], dq=s["dq"],
                                grad_dtype=s["grad"])


def run(s: dict):
    if own:
        return _own(s)
    plain = {"qkv": _plain_qkv, "qkv_grad": _plain_qkv_grad, "attn": _plain_attn, "attn_grad": _plain_attn_grad,
             "tables": _plain_tables}[s["op"]]
    return plain(s)


# --------------------------------------------------------------------------------- what it needs
def work(case: dict) -> dict:
    size = 2
    if case["op"] in ("qkv", "qkv_grad"):
        B, N, Hq, Hk, d = (case[k] for k in ("B", "N", "Hq", "Hk", "d"))
        rows, normed = B * N * (Hq + 2 * Hk), B * N * (Hq + Hk)
        # cos and sin of the positions that occur, and the positions where they are looked up
        angles = 4 * min(case["table"], B * N) * case["rot"] + 4 * B * N if case["table"] else 4 * N * case["rot"]
        bytes_ = 2 * size * rows * d + angles
        if case["op"] == "qkv_grad" and case["norm"]:
            bytes_ += size * normed * d
        return dict(bytes=bytes_, flops=(10 if case["op"] == "qkv" else 18) * normed * d)
    BH, H, W, d = (case[k] for k in ("BH", "H", "W", "d"))
    N = H * W
    if case["op"] == "tables":
        dq = {"none": 0, "f32": 4}.get(case["dq"], 2)
        out = dq or 2
        return dict(bytes=BH * N * (4 * (H + W) + (size + dq + out) * d) + (size + 4) * (2 * H + 2 * W - 2) * d,
                    flops=4 * BH * N * (H + W) * d)
    bias = 4 if case["bias"] == "f32" else 2
    if case["op"] == "attn":
        return dict(bytes=BH * N * (4 * size * d + bias * (H + W) + 4), flops=4 * BH * N * N * d)
    return dict(bytes=BH * N * (8 * size * d + (bias + 4) * (H + W) + 4), flops=10 * BH * N * N * d)


# ------------------------------------------------------------------------------- the 64-bit values
def _turn64(x: torch.Tensor, pos: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, pairs: torch.Tensor, sign: float):
    """x [rows, heads, d] in 64 bits, its pairs of columns turned by the angles of pos [rows]."""
    i, j = pairs
    c, s = cos.double()[pos].unsqueeze(1), sign * sin.double()[pos].unsqueeze(1)
    z = x.clone()
    z[:, :, i] = c * x[:, :, i] - s * x[:, :, j]
    z[:, :, j] = s * x[:, :, i] + c * x[:, :, j]
    return z


def _exact_qkv(case: dict, st: dict):
    B, N, d, rot = case["B"], case["N"], case["d"], case["rot"]
    half = torch.arange(rot // 2, device="cuda")
    pairs = torch.stack((2 * half, 2 * half + 1) if case["interleaved"] else (half, half + rot // 2))
    pos = (torch.arange(N, device="cuda").repeat(B) if st["pos"] is None else st["pos"].reshape(-1).long())
    res = []
    for b0 in range(0, B, 4):   # a few sequences at a time
        rows = slice(b0 * N, min(B, b0 + 4) * N)
        for x, w, dz in ((st["q"], st["qw"], st.get("dq")), (st["k"], st["kw"], st.get("dk"))):
            h = x.shape[2]
            v = x[b0:b0 + 4].double().reshape(-1, h, d)
            inv = (v.square().sum(-1, keepdim=True) / d + EPS).pow(-0.5)
            if case["op"] == "qkv":
                y = v if w is None else v * inv * w.double()
                y = _turn64(y, pos[rows], st["cos"], st["sin"], pairs, 1.0) if rot else y
                res.append(y.view(-1, N, h, d).permute(0, 2, 1, 3).reshape(-1, N, d))
                continue
            g = dz.view(B, h, N, d)[b0:b0 + 4].double().permute(0, 2, 1, 3).reshape(-1, h, d)
            g = _turn64(g, pos[rows], st["cos"], st["sin"], pairs, -1.0) if rot else g
            if w is None:
                res.append((g.view(-1, N, h, d), None))
                continue
            gw = (g * v * inv).sum((0, 1))
            g = g * w.double()
            g = g * inv - v * inv.pow(3) * ((g * v).sum(-1, keepdim=True) / d)
            res.append((g.view(-1, N, h, d), gw))
    if case["op"] == "qkv":
        v = st["v"].double().permute(0, 2, 1, 3).reshape(-1, N, d)
        return torch.cat(res[0::2]), torch.cat(res[1::2]), v
    dv = st["dv"].double().view(B, -1, N, d).permute(0, 2, 1, 3)
    one = [torch.cat([r[0] for r in res[k::2]]) for k in (0, 1)]
    gws = [None if res[k][1] is None else torch.stack([r[1] for r in res[k::2]]).sum(0) for k in (0, 1)]
    return one[0], one[1], dv, gws[0], gws[1]


def _exact_attn(case: dict, st: dict):
    H, W, c = case["H"], case["W"], st["scale"]
    res = []
    for b in range(case["BH"]):   # one problem at a time
        q, k, v = (st[n][b].double() for n in ("q", "k", "v"))
        rh, rw = st["rel_h"][b].double(), st["rel_w"][b].double()
        x = c * (q @ k.T) + rh.repeat_interleave(W, 1) + rw.repeat(1, H)
        if case["op"] == "attn":
            m = torch.where(x > -1e30, x, -math.inf).logsumexp(1)
            some = m > -math.inf
            p = (x - torch.where(some, m, 0.0)[:, None]).exp() * some[:, None]
            res.append((p @ v, m / math.log(2)))
            continue
        m = st["lse"][b].double() * math.log(2)
        some = m > -math.inf
        p = (x - torch.where(some, m, 0.0)[:, None]).exp() * some[:, None]
        do = st["dout"][b].double()
        g = p * (do @ v.T - (do * st["out"][b].double()).sum(1, keepdim=True))
        gg = g.view(-1, H, W)
        res.append((c * (g @ k), c * (g.T @ q), p.T @ do, gg.sum(2), gg.sum(1)))
    return tuple(torch.stack(list(r)) for r in zip(*res))


def _exact_tables(case: dict, st: dict):
    BH, H, W, d = (case[k] for k in ("BH", "H", "W", "d"))
    th, tw = st["th"].double(), st["tw"].double()
    gth, gtw = torch.zeros_like(th), torch.zeros_like(tw)
    dq = torch.zeros(BH, H, W, d, dtype=torch.float64, device="cuda")
    q = st["q"].double().view(BH, H, W, d)
    gh, gw = st["drel_h"].double().view(BH, H, W, H), st["drel_w"].double().view(BH, H, W, W)
    for a in range(H):   # the table rows a + H - 1 down to a
        rows = slice(a, a + H)
        g = gh[:, a].flip(-1)
        dq[:, a] += g @ th[rows]
        gth[rows] += g.reshape(-1, H).T @ q[:, a].reshape(-1, d)
    for a in range(W):
        rows = slice(a, a + W)
        g = gw[:, :, a].flip(-1)
        dq[:, :, a] += g @ tw[rows]
        gtw[rows] += g.reshape(-1, W).T @ q[:, :, a].reshape(-1, d)
    dq = dq.view(BH, H * W, d)
    return (dq if st["dq"] is None else dq + st["dq"].double()), gth, gtw


def exact(case: dict, seed: int):
    st = prepare(case, seed)
    make = {"qkv": _exact_qkv, "qkv_grad": _exact_qkv, "attn": _exact_attn, "attn_grad": _exact_attn,
            "tables": _exact_tables}[case["op"]]
    return make(case, st)
