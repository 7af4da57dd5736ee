"""ctypes binding of the entry points in ``include/dera_block.h`` (argument marshalling only).

The rest of an encoder block around the attention: :func:`layer_norm`, :func:`linear` (bias, activation
and residual in one kernel, reading the attention's heads as they lie), :func:`activation_backward`,
and the backward of each.  As in ``api`` and ``train``: shapes are checked, pointers and the stream are
passed on, and error codes become exceptions; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import api
from .api import DERA_F32, _check, _fits, _ptr
from .train import _dtype, _launch_stream, _pack_heads, _same, _scratch, _size, _want

HEADER = os.path.join(os.path.dirname(api.HEADER), "dera_block.h")

# ``dera_activation``
ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "quick_gelu": 4, "silu": 5}


def declare(lib: ctypes.CDLL) -> None:
    """Signatures of the entry points (called by ``api.load_library``)."""
    vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    szp = ctypes.POINTER(sz)
    for name, args in {
        "dera_layer_norm": [vp] * 6 + [i, i, ll, f, i, i, i, vp],
        "dera_layer_norm_backward_workspace_size": [i, i, szp],
        "dera_layer_norm_backward": [vp] * 9 + [i, i, ll, i, i, i, i, vp, sz, vp],
        "dera_linear": [vp] * 6 + [i] * 9 + [vp],
        "dera_linear_backward_workspace_size": [i] * 5 + [szp],
        "dera_linear_backward": [vp] * 7 + [i] * 9 + [vp, sz, vp],
        "dera_activation_backward": [vp] * 3 + [ll, i, i, i, i, vp],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i


def _activation(name: str | None) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}: one of {list(ACTIVATIONS)}")
    return code


# ------------------------------------------------------------------------------------- layer norm
def _norm_rows(x: torch.Tensor) -> tuple[int, int, int]:
    """(rows, columns, elements from row to row) of [..., C]."""
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    C = x.shape[-1]
    rows = x.numel() // C if C else 0
    _fits(rows | C)
    if x.is_contiguous() or rows == 0:
        return rows, C, C
    if x.stride(-1) != 1 and C > 1:
        raise ValueError("x: the last dimension must be contiguous")
    try:
        return rows, C, x.view(rows, C).stride(0)
    except RuntimeError:
        raise ValueError("x: its rows must lie at one stride") from None


def _norm_params(weight, bias, C: int, dtypes: tuple) -> int:
    """The weights' dtype code after the checks that forward and backward share."""
    if weight is None:
        if bias is not None:
            raise ValueError("a bias needs a weight")
        return DERA_F32
    if weight.dtype not in dtypes:
        raise TypeError(f"the weight must be one of {dtypes}")
    _same(weight, (C,), weight.dtype, "weight")
    _same(bias, (C,), weight.dtype, "bias")
    return _dtype(weight.dtype)


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               eps: float = 1e-6, out_dtype: torch.dtype | None = None, stream=None
               ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm of the last dimension via ``dera_layer_norm``: ``(y, mean, rstd)``.

    x ``[..., C]``, fp16, bf16 or fp32, its rows at one stride; weight and bias ``[C]``, fp32 or of x's or y's
    dtype (None: 1 and 0).  y is contiguous in ``out_dtype`` (default x's; fp32 or, for an fp32 x, any); mean and
    rstd ``[...]`` fp32 are what :func:`layer_norm_backward` takes."""
    rows, C, xs = _norm_rows(x)
    od = out_dtype or x.dtype
    wcode = _norm_params(weight, bias, C, (torch.float32, x.dtype, od))
    dev = x.device
    y = torch.empty(x.shape, dtype=od, device=dev)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    _check(api.load_library().dera_layer_norm(
        x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, C, xs, eps,
        _dtype(x.dtype), wcode, _dtype(od), _launch_stream(dev, stream)))
    return y, mean, rstd


def layer_norm_backward_workspace_size(rows: int, cols: int) -> int:
    """Scratch bytes of :func:`layer_norm_backward` on the current device."""
    return _size("dera_layer_norm_backward_workspace_size", rows, cols)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: torch.Tensor | None = None, *, dres: torch.Tensor | None = None,
                        grad_dtype: torch.dtype | None = None, stream=None, workspace: torch.Tensor | None = None):
    """Gradients of :func:`layer_norm` via ``dera_layer_norm_backward``: ``(dx, dweight, dbias)``.

    x and weight are the forward's, mean and rstd what it returned, dy the gradient of y (contiguous).  ``dres``, if
    given, is a gradient that reaches x past the norm (of the residual stream, in ``grad_dtype``), to which dx is added.
    dx comes contiguous in ``grad_dtype`` (default fp32), dweight and dbias in fp32 (None without a weight)."""
    rows, C, xs = _norm_rows(x)
    gd = grad_dtype or (torch.float32 if dres is None else dres.dtype)
    wcode = _norm_params(weight, None, C, (torch.float32, x.dtype, dy.dtype))
    _want(dy, x.shape, "dy")
    _same(mean, x.shape[:-1], torch.float32, "mean")
    _same(rstd, x.shape[:-1], torch.float32, "rstd")
    _same(dres, x.shape, gd, "dres")
    dev = x.device
    dx = torch.empty(x.shape, dtype=gd, device=dev)
    st = _launch_stream(dev, stream)
    dw = db = keep = ws = None
    ws_bytes = 0
    if weight is not None:
        dw = torch.empty(C, dtype=torch.float32, device=dev)
        db = torch.empty(C, dtype=torch.float32, device=dev)
        keep, ws, ws_bytes = _scratch(dev, stream, st, workspace, "dera_layer_norm_backward_workspace_size", rows, C)
    _check(api.load_library().dera_layer_norm_backward(
        dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(weight), _ptr(dres), dx.data_ptr(), _ptr(dw),
        _ptr(db), rows, C, xs, _dtype(x.dtype), wcode, _dtype(dy.dtype), _dtype(gd), ws, ws_bytes, st))
    return dx, dw, db


# ----------------------------------------------------------------------------------------- linear
def _tokens(x: torch.Tensor, K: int, name: str) -> tuple[int, int, int, int]:
    """(B, N, heads, head_dim) of tokens of K features: [K], [N, K], [B, N, K] or [B, N, heads, head_dim]."""
    shape = x.shape
    if len(shape) == 4 and shape[2] * shape[3] == K:
        return tuple(shape)
    if not 1 <= len(shape) <= 3 or shape[-1] != K:
        raise ValueError(f"{name}: expected up to three dimensions, the last of {K}, or [B, N, heads, d] with as many "
                         f"features, got {tuple(shape)}")
    return (1, 1, *shape[:-1])[-2:] + (1, K)


def _out_shape(x: torch.Tensor, out: int) -> tuple:
    return (*x.shape[:2], out) if x.dim() == 4 else (*x.shape[:-1], out)


def _token_heads(x: torch.Tensor, name: str) -> bytes:
    """The ``dera_heads`` of tokens."""
    st = x.stride()
    if st[-1] != 1 and x.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    sb, sn, sh = st[:3] if len(st) == 4 else (0, 0, *st[:-1])[-2:] + (0,)
    return _pack_heads(x.data_ptr(), sb, sn, sh)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *, activation: str | None = None,
           residual: torch.Tensor | None = None, keep_pre: bool = False, out_dtype: torch.dtype | None = None, stream=None):
    """``act(x weight^T + bias) + residual`` via ``dera_linear``.

    x ``[K]``, ``[N, K]`` or ``[B, N, K]`` with any strides that are multiples of 8, or ``[B, N, heads, d]`` with
    ``heads * d = K`` (four dimensions are always these): what the attention returns is
    ``out.view(B, heads, N, d).transpose(1, 2)``, read as it lies.
    weight ``[out_features, K]`` of x's dtype (fp16 or bf16), bias ``[out_features]`` fp32 or x's.  ``activation``: None,
    "relu", "gelu", "gelu_tanh", "quick_gelu" or "silu".  ``residual``: of the output's shape and dtype.  Returns y
    ``[..., out_features]`` (``[B, N, out_features]`` from heads) in ``out_dtype`` (default x's; fp32), with ``keep_pre``
    ``(y, pre)``: what the activation was given, in x's dtype."""
    if weight.dim() != 2:
        raise ValueError("weight must be [out_features, K]")
    out, K = weight.shape
    B, N, heads, d = _tokens(x, K, "x")
    _fits(B | N | heads | d | out)
    dt, dev = x.dtype, x.device
    od = out_dtype or dt
    _same(weight, (out, K), dt, "weight")
    if bias is not None and bias.dtype not in (dt, torch.float32):
        raise TypeError("the bias must be float32 or of x's dtype")
    size = _out_shape(x, out)
    if bias is not None:
        _want(bias, (out,), "bias")
    _same(residual, size, od, "residual")
    y = torch.empty(size, dtype=od, device=dev)
    pre = torch.empty(size, dtype=dt, device=dev) if keep_pre else None
    _check(api.load_library().dera_linear(
        _token_heads(x, "x"), weight.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(pre), B, N, heads, d, out,
        _activation(activation), _dtype(dt), DERA_F32 if bias is None else _dtype(bias.dtype), _dtype(od),
        _launch_stream(dev, stream)))
    return (y, pre) if keep_pre else y


def linear_backward_workspace_size(B: int, N: int, heads: int, head_dim: int, out_features: int) -> int:
    """Scratch bytes of :func:`linear_backward` on the current device."""
    return _size("dera_linear_backward_workspace_size", B, N, heads, head_dim, out_features)


def linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *, input_pre: torch.Tensor | None = None,
                    input_activation: str | None = None, input_grad: bool = True, weight_grad: bool = True,
                    bias_grad: bool = True, grad_dtype: torch.dtype | None = None,
                    weight_grad_dtype: torch.dtype | None = None, stream=None, workspace: torch.Tensor | None = None):
    """Gradients of ``x weight^T + bias`` via ``dera_linear_backward``: ``(dx, dweight, dbias)``.

    dy is the gradient of the sum before any activation (of the residual, too), contiguous, of x's dtype; x and weight are
    the forward's.  With ``input_activation`` and ``input_pre`` (of x's shape and dtype, what the layer before kept) x is taken
    as that activation's value and dx is the gradient of ``input_pre``.  dx has x's shape (and its layout where it is
    dense) in ``grad_dtype`` (default fp32), dweight comes in ``weight_grad_dtype`` (default fp32), dbias in fp32; None for
    what ``input_grad``, ``weight_grad`` and ``bias_grad`` leave out."""
    if weight.dim() != 2:
        raise ValueError("weight must be [out_features, K]")
    out, K = weight.shape
    B, N, heads, d = _tokens(x, K, "x")
    _fits(B | N | heads | d | out)
    dt, dev = x.dtype, x.device
    gd, wd = grad_dtype or torch.float32, weight_grad_dtype or torch.float32
    _same(weight, (out, K), dt, "weight")
    _same(dy, _out_shape(x, out), dt, "dy")
    if (input_pre is None) != (input_activation is None):
        raise ValueError("input_pre and input_activation go together")
    if input_pre is not None and (input_pre.shape != x.shape or input_pre.dtype != dt):
        raise ValueError(f"input_pre must have x's shape and dtype, got {tuple(input_pre.shape)} {input_pre.dtype}")
    dx = dw = db = keep = ws = None
    ws_bytes = 0
    if input_grad:
        dx = torch.empty_like(x, dtype=gd)
    if weight_grad:
        dw = torch.empty((out, K), dtype=wd, device=dev)
    if bias_grad:
        db = torch.empty(out, dtype=torch.float32, device=dev)
    st = _launch_stream(dev, stream)
    if weight_grad or bias_grad:
        keep, ws, ws_bytes = _scratch(dev, stream, st, workspace, "dera_linear_backward_workspace_size", B, N, heads, d, out)
    _check(api.load_library().dera_linear_backward(
        dy.data_ptr(), _token_heads(x, "x"), weight.data_ptr(),
        None if input_pre is None else _token_heads(input_pre, "input_pre"),
        None if dx is None else _token_heads(dx, "dx"), _ptr(dw), _ptr(db), B, N, heads, d, out,
        _activation(input_activation), _dtype(dt), _dtype(gd), _dtype(wd), ws, ws_bytes, st))
    return dx, dw, db


def activation_backward(dy: torch.Tensor, pre: torch.Tensor, activation: str, *, grad_dtype: torch.dtype | None = None,
                        stream=None) -> torch.Tensor:
    """``dy * act'(pre)`` via ``dera_activation_backward``: from the gradient of an activation's value to that of what it
    was given, where no :func:`linear_backward` takes it through (``input_activation``).

    dy and pre of one shape, contiguous; dy fp32 or of pre's dtype; the result in ``grad_dtype`` (default fp32)."""
    _want(dy, pre.shape, "dy")
    _want(pre, pre.shape, "pre")
    code = _activation(activation)
    if not code:
        raise ValueError("activation_backward needs an activation")
    gd = grad_dtype or torch.float32
    dpre = torch.empty(pre.shape, dtype=gd, device=pre.device)
    _check(api.load_library().dera_activation_backward(
        dy.data_ptr(), pre.data_ptr(), dpre.data_ptr(), pre.numel(), code, _dtype(pre.dtype), _dtype(dy.dtype), _dtype(gd),
        _launch_stream(pre.device, stream)))
    return dpre
