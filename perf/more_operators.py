"""The encoder block's other operators, as they are measured.

Five kinds of case, each one pass of an operator:

  norm         layer_norm: the rows of the residual stream normed, with their statistics
  norm_grad    layer_norm_backward: dx (with the residual's gradient added), dweight, dbias
  linear       linear: x W^T with bias, activation and residual
  linear_grad  linear_backward: dx (on through the activation that x came from), dweight, dbias
  act_grad     activation_backward: the gradient of what an activation was given

``own`` selects between the plain form (elementary torch operations in 32 bits) and the library's
entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "quick_gelu", "silu"]


# ------------------------------------------------------------------------------------------ cases
def _norm(name: str, op: str, rows: int, C: int, **kw) -> dict:
    return dict(name=name, op=op, rows=rows, C=C, **(dict(dtype="bf16", y="bf16", affine=True, res=False) | kw))


def _linear(name: str, op: str, B: int, N: int, K: int, out: int, **kw) -> dict:
    """B * N tokens, K features in (by heads of `d` where d > 0, as the attention leaves them), `out` features out."""
    base = dict(dtype="bf16", d=0, bias=True, act="none", res=False, pre=False, y="bf16", input_act="none", dw="f32")
    return dict(name=name, op=op, B=B, N=N, K=K, out=out, **(base | kw))


def listed() -> list[dict]:
    return [
        # one new token in each of 32 sequences: latency counts
        _norm("norm_token", "norm", 32, 1024),
        # eight 64x64 encoders 2048 wide: bandwidth
        _norm("norm_wide64", "norm", 8 * 4096, 2048, dtype="f16", y="f16"),
        # the windowed blocks of one image, 12 heads of 64 wide; the residual's gradient joins
        _norm("norm_grad_window14", "norm_grad", 25 * 196, 768, res=True),
        # eight images whose residual stream is kept in 32 bits
        _norm("norm_grad_stream64", "norm_grad", 8 * 4096, 1024, dtype="f32", y="bf16", res=True),
        # one new token in each of 32 sequences through the perceptron's first layer: latency counts
        _linear("linear_token", "linear", 32, 1, 1024, 4096, act="gelu"),
        # the packed projection of one image's windows, 12 heads of 64
        _linear("linear_window14", "linear", 25, 196, 768, 2304),
        # eight images in training: the first layer keeps what its activation was given
        _linear("linear_mlp64", "linear", 8, 4096, 1024, 4096, act="gelu", pre=True),
        # the output projection straight from the attention's heads, onto the residual stream
        _linear("linear_heads64", "linear", 8, 4096, 2048, 2048, d=128, res=True),
        # the second layer's gradients for eight images, on to what the first one's activation was given
        _linear("linear_grad_mlp64", "linear_grad", 8, 4096, 4096, 1024, input_act="gelu"),
        # the output projection's gradients for images of an odd size, from and to the attention's heads
        _linear("linear_grad_ragged", "linear_grad", 3, 37 * 37, 768, 1000, dtype="f16", y="f16", d=64),
        # a perceptron's last activation, one image's windows
        _linear("act_grad_window14", "act_grad", 25, 196, 0, 768, act="silu"),
        # the same for eight images, the gradient in 32 bits
        _linear("act_grad_wide64", "act_grad", 8, 4096, 0, 2048, dtype="f16", act="quick_gelu", y="f32"),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng) -> dict:
    op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "linear_grad", "act_grad"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("norm", "norm_grad"):
        x = rng.choice([dtype, dtype, "f32"])
        C = _log_int(rng, 1, 8192)
        rows = _log_int(rng, 1, min(32768, 32768 * 1024 // C))
        case = _norm("", op, rows, C, dtype=x, y=dtype if x == "f32" else rng.choice([x, x, "f32"]),
                     affine=rng.random() < 0.8, res=op == "norm_grad" and rng.random() < 0.5)
    elif op == "act_grad":
        out = _log_int(rng, 1, 8192)
        B = _log_int(rng, 1, 32)
        N = _log_int(rng, 1, max(1, min(4096, 32768 * 2048 // (out * B))))
        case = _linear("", op, B, N, 0, out, dtype=dtype, y=rng.choice([dtype, "f32"]), act=rng.choice(ACTIVATIONS[1:]))
    else:
        most = 2 * 32768 * 1024 * 4096 if op == "linear" else 32768 * 1024 * 4096
        d = rng.choice([0, 0, 64, 128])
        K = d * _log_int(rng, 1, 4096 // d) if d else 8 * _log_int(rng, 1, 1024)
        out = 8 * _log_int(rng, 1, 1024)
        tokens = _log_int(rng, 1, max(1, min(40000, most // (K * out) // 2)))
        B = _log_int(rng, 1, min(tokens, 32))
        case = _linear("", op, B, max(1, tokens // B), K, out, d=d, dtype=dtype, y=rng.choice([dtype, dtype, "f32"]))
        if op == "linear":
            case |= dict(act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.8, res=rng.random() < 0.4,
                         pre=rng.random() < 0.4)
        else:
            case |= dict(input_act=rng.choice(["none"] + ACTIVATIONS), dw=rng.choice(["f32", "f32", dtype]))
    del case["name"]
    return case


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed: int) -> torch.Generator:
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, s: float = 1.0, dtype=torch.float32) -> torch.Tensor:
    return (torch.randn(*shape, generator=g, device="cuda") * s).to(dtype)


def _prepare_norm(case: dict, g) -> dict:
    rows, C, t, y = case["rows"], case["C"], DTYPES[case["dtype"]], DTYPES[case["y"]]
    # a residual stream: rows of unequal size off zero, channels of unequal size, some far larger
    chan = torch.exp(0.5 * torch.randn(C, generator=g, device="cuda"))
    chan = chan.where(torch.rand(C, generator=g, device="cuda") < 0.99, 10 * chan)
    size = torch.exp(0.3 * torch.randn(rows, 1, generator=g, device="cuda"))
    x = torch.randn(rows, C, generator=g, device="cuda").mul_(chan).add_(0.5).mul_(size).to(t)
    s = dict(x=x, weight=None, bias=None, y=y)
    if case["affine"]:
        s["weight"], s["bias"] = _randn(g, C, s=0.2).add_(1), _randn(g, C, s=0.2)
    if case["op"] == "norm_grad":
        # what the forward pass of the step left behind
        xf = x.double() if C * rows < 1 << 22 else x.float()
        mean = xf.mean(-1)
        s["mean"] = mean.float()
        s["rstd"] = ((xf - mean[:, None]).square_().mean(-1) + EPS).rsqrt().float()
        s["dy"] = _randn(g, rows, C, s=0.02, dtype=y)
        s["dres"] = _randn(g, rows, C, s=0.02, dtype=t) if case["res"] else None
    return s


def _features(case: dict, g, t) -> torch.Tensor:
    """Tokens as a norm leaves them: [B, N, K], or [B, N, heads, d] over the attention's [B * heads, N, d]."""
    B, N, K, d = (case[k] for k in ("B", "N", "K", "d"))
    if d:
        return torch.randn(B, K // d, N, d, generator=g, device="cuda", dtype=t).transpose(1, 2)
    chan = 0.5 + torch.rand(K, generator=g, device="cuda")
    return torch.randn(B, N, K, generator=g, device="cuda", dtype=t).mul_(chan.to(t))


def _prepare_linear(case: dict, g) -> dict:
    B, N, K, out, t = case["B"], case["N"], case["K"], case["out"], DTYPES[case["dtype"]]
    # rows of very different size, as a loss gives them
    size = 0.05 * torch.exp(torch.randn(B, N, 1, generator=g, device="cuda"))
    if case["op"] == "act_grad":
        return dict(pre=_randn(g, B, N, out, dtype=t), act=case["act"], y=DTYPES[case["y"]],
                    dy=torch.randn(B, N, out, generator=g, device="cuda", dtype=t).mul_(size.to(t)))
    s = dict(weight=_randn(g, out, K, s=K ** -0.5, dtype=t), act=case["act"], y=DTYPES[case["y"]], bias=None,
             input_act=case["input_act"], input_pre=None)
    x = _features(case, g, t)
    if case["op"] == "linear":
        s["x"], s["keep"] = x, case["pre"]
        s["bias"] = _randn(g, out, s=0.3, dtype=t) if case["bias"] else None
        s["res"] = _randn(g, B, N, out, dtype=s["y"]) if case["res"] else None
        return s
    # what the forward pass of the step left behind
    if case["input_act"] != "none":
        s["input_pre"], x = x, _activate(x.float(), case["input_act"]).to(t)
    s["x"], s["dw"] = x, DTYPES[case["dw"]]
    s["dy"] = torch.randn(B, N, out, generator=g, device="cuda", dtype=t).mul_(size.to(t))
    return s


def prepare(case: dict, seed: int) -> dict:
    make = _prepare_norm if case["op"] in ("norm", "norm_grad") else _prepare_linear
    s = make(case, _gen(seed))
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------------------------- plain forms
def _sigmoid(z: torch.Tensor) -> torch.Tensor:
    return 1.0 / (1.0 + torch.exp(-z))


def _activate(u: torch.Tensor, act: str) -> torch.Tensor:
    if act == "none":
        return u
    if act == "relu":
        return u.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * u * torch.erfc(u * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return u * _sigmoid(2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u * u * u))
    return u * _sigmoid(1.702 * u if act == "quick_gelu" else u)


def _slope(u: torch.Tensor, act: str) -> torch.Tensor:
    """The activation's derivative."""
    if act == "relu":
        return (u > 0).to(u.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(u * -math.sqrt(0.5)) + u * torch.exp(-0.5 * u * u) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        sg = _sigmoid(c * (u + 0.044715 * u * u * u))
        return sg + u * sg * (1 - sg) * c * (1 + 3 * 0.044715 * u * u)
    c = 1.702 if act == "quick_gelu" else 1.0
    sg = _sigmoid(c * u)
    return sg + c * u * sg * (1 - sg)


def _plain_norm(s: dict):
    x = s["x"].float()
    mean = x.mean(-1)
    x = x - mean[:, None]
    rstd = torch.rsqrt((x * x).mean(-1) + EPS)
    y = x * rstd[:, None]
    if s["weight"] is not None:
        y = y * s["weight"] + s["bias"]
    return y.to(s["y"]), mean, rstd


def _plain_norm_grad(s: dict):
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy if s["weight"] is None else dy * s["weight"]
    dx = s["rstd"][:, None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    if s["weight"] is None:
        return dx.to(s["x"].dtype), None, None
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _rows(x: torch.Tensor) -> torch.Tensor:
    """[tokens, features] in 32 bits, heads side by side."""
    return x.float().reshape(x.shape[0] * x.shape[1], -1)


def _plain_linear(s: dict):
    x = s["x"]
    u = _rows(x) @ s["weight"].float().T
    if s["bias"] is not None:
        u = u + s["bias"].float()
    u = u.view(x.shape[0], x.shape[1], -1)
    y = _activate(u, s["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return (y.to(s["y"]), u.to(x.dtype)) if s["keep"] else y.to(s["y"])


def _plain_linear_grad(s: dict):
    x, g = s["x"], _rows(s["dy"])
    dx = (g @ s["weight"].float()).view(x.shape)
    if s["input_pre"] is not None:
        dx = dx * _slope(s["input_pre"].float(), s["input_act"])
    return dx.to(s["y"]), (g.T @ _rows(x)).to(s["dw"]), g.sum(0)


def _plain_act_grad(s: dict):
    return (s["dy"].float() * _slope(s["pre"].float(), s["act"])).to(s["y"])


# ------------------------------------------------------------------------------------ one pass
def _name(act: str) -> str | None:
    return None if act == "none" else act


def _own(s: dict):
    import relative_position_bias_gb300 as rpb

    if s["op"] == "norm":
        return rpb.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, out_dtype=s["y"])
    if s["op"] == "norm_grad":
        return rpb.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], dres=s["dres"],
                                       grad_dtype=s["x"].dtype)
    if s["op"] == "linear":
        return rpb.linear(s["x"], s["weight"], s["bias"], activation=_name(s["act"]), residual=s["res"],
                          keep_pre=s["keep"], out_dtype=s["y"])
    if s["op"] == "act_grad":
        return rpb.activation_backward(s["dy"], s["pre"], s["act"], grad_dtype=s["y"])
    return rpb.linear_backward(s["dy"], s["x"], s["weight"], input_pre=s["input_pre"],
                               input_activation=_name(s["input_act"]), grad_dtype=s["y"], weight_grad_dtype=s["dw"])


def run(s: dict):
    if own:
        return _own(s)
    plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "linear": _plain_linear,
             "linear_grad": _plain_linear_grad, "act_grad": _plain_act_grad}[s["op"]]
    return plain(s)


# --------------------------------------------------------------------------------- what it needs
def work(case: dict) -> dict:
    size = {"bf16": 2, "f16": 2, "f32": 4}
    x, y = size[case["dtype"]], size[case["y"]]
    if case["op"] in ("norm", "norm_grad"):
        n, C = case["rows"] * case["C"], case["C"]
        if case["op"] == "norm":
            return dict(bytes=n * (x + y) + 8 * case["rows"] + 8 * C * case["affine"], flops=8 * n)
        return dict(bytes=n * (2 * x + y + x * case["res"]) + 8 * case["rows"] + 12 * C * case["affine"], flops=16 * n)
    M, K, out = case["B"] * case["N"], case["K"], case["out"]
    if case["op"] == "act_grad":
        return dict(bytes=M * out * (2 * x + y), flops=15 * M * out)
    if case["op"] == "linear":
        return dict(bytes=x * (M * K + K * out + out * case["bias"]) + M * out * (y + y * case["res"] + x * case["pre"]),
                    flops=2 * M * K * out)
    acts = x * M * K * (case["input_act"] != "none")
    return dict(bytes=x * (M * K + M * out + K * out) + acts + y * M * K + size[case["dw"]] * K * out + 4 * out,
                flops=4 * M * K * out)


# ------------------------------------------------------------------------------- the 64-bit values
def _act64(u: torch.Tensor, act: str) -> torch.Tensor:
    if act == "relu":
        return torch.where(u > 0, u, 0.0)
    if act == "gelu":
        return u * torch.special.ndtr(u)
    if act == "gelu_tanh":
        return 0.5 * u * (1 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u.pow(3))))
    return u if act == "none" else u * torch.special.expit({"quick_gelu": 1.702, "silu": 1.0}[act] * u)


def _slope64(u: torch.Tensor, act: str) -> torch.Tensor:
    if act in ("none", "relu"):
        return torch.ones_like(u) if act == "none" else torch.heaviside(u, torch.zeros((), dtype=u.dtype, device=u.device))
    if act == "gelu":
        return torch.special.ndtr(u) + u * (-u.square() / 2).exp() / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        b = math.sqrt(2 / math.pi)
        th = torch.tanh(b * (u + 0.044715 * u.pow(3)))
        return 0.5 * (1 + th) + 0.5 * u * (1 - th.square()) * b * (1 + 0.134145 * u.square())
    b = {"quick_gelu": 1.702, "silu": 1.0}[act]
    return torch.special.expit(b * u) * (1 + b * u * torch.special.expit(-b * u))


def _exact_norm(case: dict, st: dict):
    res, C = [], case["C"]
    gw = gb = torch.zeros(C, dtype=torch.float64, device="cuda")
    w = None if st["weight"] is None else st["weight"].double()
    for r in range(0, case["rows"], 4096):   # some rows at a time
        part = slice(r, r + 4096)
        x = st["x"][part].double()
        if case["op"] == "norm":
            var, mu = torch.var_mean(x, -1, correction=0, keepdim=True)
            inv = (var + EPS).pow(-0.5)
            h = inv * (x - mu)
            res.append((h if w is None else h * w + st["bias"].double(), mu[:, 0], inv[:, 0]))
            continue
        inv, dy = st["rstd"][part, None].double(), st["dy"][part].double()
        h = inv * (x - st["mean"][part, None].double())
        gw, gb = gw + torch.einsum("rc,rc->c", dy, h), gb + dy.sum(0)
        q = dy if w is None else dy * w
        dx = inv * (q - (q.sum(-1, keepdim=True) + h * torch.einsum("rc,rc->r", q, h)[:, None]) / C)
        res.append((dx if st["dres"] is None else dx + st["dres"][part].double(),))
    parts = tuple(torch.cat(list(p)) for p in zip(*res))
    if case["op"] == "norm":
        return parts
    return (parts[0], None, None) if w is None else (parts[0], gw, gb)


def _exact_linear(case: dict, st: dict):
    w, K = st["weight"].double(), case["K"]
    x = st["x"].reshape(case["B"] * case["N"], K)
    shape = (case["B"], case["N"], -1)
    if case["op"] == "linear":
        ys, us = [], []
        for r in range(0, x.shape[0], 4096):
            u = torch.einsum("mk,nk->mn", x[r:r + 4096].double(), w)
            if st["bias"] is not None:
                u += st["bias"].double()
            ys.append(_act64(u, case["act"]))
            us.append(u)
        y = torch.cat(ys).view(shape)
        if st["res"] is not None:
            y = y + st["res"].double()
        return (y, torch.cat(us).view(shape)) if case["pre"] else y
    g = st["dy"].reshape(-1, case["out"]).double()
    dw, dxs = torch.zeros_like(w), []
    ip = None if st["input_pre"] is None else st["input_pre"].reshape(-1, K)
    for r in range(0, x.shape[0], 4096):
        part = slice(r, r + 4096)
        dw += torch.einsum("mn,mk->nk", g[part], x[part].double())
        dx = torch.einsum("mn,nk->mk", g[part], w)
        dxs.append(dx if ip is None else dx * _slope64(ip[part].double(), case["input_act"]))
    return torch.cat(dxs).view(st["x"].shape), dw, g.sum(0)


def exact(case: dict, seed: int):
    st = prepare(case, seed)
    if case["op"] == "act_grad":
        return _slope64(st["pre"].double(), case["act"]) * st["dy"].double()
    return (_exact_norm if case["op"] in ("norm", "norm_grad") else _exact_linear)(case, st)
