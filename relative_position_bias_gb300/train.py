"""ctypes binding of the entry points in ``include/dera_train.h`` (argument marshalling only).

What a training step needs around :func:`~relative_position_bias_gb300.attention`: the heads of a
packed projection normed, rotated and laid out (:func:`qk_norm_rope`), the compact-bias attention
with its log-sum-exp (:func:`attention_lse`), and the backward of each step
(:func:`attention_backward`, :func:`project_backward`, :func:`qk_norm_rope_backward`).  As in
``api``: shapes are checked, pointers and the stream are passed on, and error codes become
exceptions; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os
import struct

import torch

from . import api
from .api import DERA_F32, _check, _expect, _fits, _ptr

HEADER = os.path.join(os.path.dirname(api.HEADER), "dera_train.h")
_CODE = api._DTYPE_CODE


# ``dera_heads``: a [B, N, heads, d] tensor by its address and strides, packed as bytes (ctypes passes their
# address; filling a ctypes array costs seven times as much)
_pack_heads = struct.Struct("=4q").pack


def declare(lib: ctypes.CDLL) -> None:
    """Signatures of the entry points (called by ``api.load_library``)."""
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    szp = ctypes.POINTER(sz)
    for name, args in {
        "dera_qk_norm_rope": [vp] * 11 + [i] * 8 + [f, i, i, vp],
        "dera_qk_norm_rope_backward_workspace_size": [i] * 5 + [szp],
        "dera_qk_norm_rope_backward": [vp] * 15 + [i] * 8 + [f] + [i] * 4 + [vp, sz, vp],
        "dera_relpos_attention_lse": [vp] * 7 + [i] * 4 + [f] + [i] * 3 + [vp, sz, vp],
        "dera_relpos_attention_backward_workspace_size": [i] * 4 + [szp],
        "dera_relpos_attention_backward": [vp] * 13 + [i] * 4 + [f] + [i] * 4 + [vp, sz, vp],
        "dera_relpos_project_backward_workspace_size": [i] * 4 + [szp],
        "dera_relpos_project_backward": [vp] * 9 + [i] * 6 + [vp, sz, vp],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i


# A call of the smallest sizes is bound by what happens before its kernels start, so these helpers
# ask PyTorch for as little as they can.
def _dtype(t: torch.dtype) -> int:
    code = _CODE.get(t)
    if code is None:
        raise TypeError(f"unsupported dtype {t}")
    return code


def _want(t: torch.Tensor, shape, name: str) -> None:
    if t.shape != shape or not t.is_contiguous():
        _expect(t, shape, name)   # says what is wrong


def _like(t: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """An empty tensor of (contiguous) t's shape."""
    return torch.empty_like(t) if t.dtype == dtype else torch.empty_like(t, dtype=dtype)


def _launch_stream(device: torch.device, stream) -> int | None:
    """Handle of the stream to launch on (the current one of `device` unless given)."""
    if stream is None and device.type == "cuda":
        return torch._C._cuda_getCurrentRawStream(device.index)
    return api._stream(device, stream)


@functools.lru_cache(maxsize=256)
def _size_on(device_index: int, entry: str, *sizes: int) -> int:
    """What a workspace-size entry says on a device (a function of the sizes and the device alone)."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device_index):
        _check(getattr(api.load_library(), entry)(*sizes, ctypes.byref(n)))
    return n.value


def _size(entry: str, *sizes: int) -> int:
    """The same on the current device, if there is one."""
    _fits(functools.reduce(operator.or_, sizes))
    n = ctypes.c_size_t(0)
    _check(getattr(api.load_library(), entry)(*sizes, ctypes.byref(n)))
    return n.value


def _scratch(device: torch.device, stream, handle, workspace: torch.Tensor | None, entry: str, *sizes: int) -> tuple:
    """(tensor to keep alive, pointer, bytes) of one call's scratch: the caller's, or a new buffer
    of the launching stream."""
    if workspace is None:
        if device.type != "cuda":
            return None, None, 0
        need = _size_on(device.index, entry, *sizes)
        if need == 0:
            return None, None, 0
        workspace = (torch.empty(need, dtype=torch.uint8, device=device) if stream is None
                     else api._scratch_on(need, device, int(handle or 0)))
        return workspace, workspace.data_ptr(), need
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ------------------------------------------------------------------------ norms, rotation, layout
def _heads(t: torch.Tensor | None, shape, name: str) -> bytes | None:
    """The ``dera_heads`` of a tensor (None: none)."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    sb, st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return _pack_heads(t.data_ptr(), sb, st, sh)


def _same(t: torch.Tensor | None, shape: tuple, dtype, name: str) -> None:
    if t is None:
        return
    _want(t, shape, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _qk_common(q, k, v, q_weight, k_weight, cos, sin, positions):
    """Sizes and the checks that forward and backward share:
    (B, N, q heads, kv heads, d, rotary_dim, table rows, weight dtype code)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, N, heads, d]")
    B, N, hq, d = q.shape
    hk = k.shape[2]
    if k.dtype != q.dtype or (v is not None and v.dtype != q.dtype):
        raise TypeError("q, k and v must share a dtype")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    wcode = DERA_F32
    if q_weight is not None:
        if q_weight.dtype not in (q.dtype, torch.float32):
            raise TypeError("the weights must be float32 or of q's dtype")
        _same(q_weight, (d,), q_weight.dtype, "q_weight")
        _same(k_weight, (d,), q_weight.dtype, "k_weight")
        wcode = _dtype(q_weight.dtype)
    rot = rows = 0
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [rows, rotary_dim / 2]")
        rows, rot = cos.shape[0], 2 * cos.shape[1]
        _same(cos, (rows, rot // 2), torch.float32, "cos")
        _same(sin, (rows, rot // 2), torch.float32, "sin")
        _same(positions, (B, N), torch.int32, "positions")
    elif positions is not None:
        raise ValueError("positions need cos and sin")
    _fits(B | N | hq | hk | d | rot | rows)
    return B, N, hq, hk, d, rot, rows, wcode


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor | None = None, *,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                 cos: torch.Tensor | None = None, sin: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False, stream=None):
    """Per-head norms of q and k and their rotation by position, via ``dera_qk_norm_rope``.

    q ``[B, N, q_heads, d]``, k and v ``[B, N, kv_heads, d]`` in token order with any strides that keep
    rows whole (slices of a packed projection as they lie).  Returns ``(q_out, k_out)``, or
    ``(q_out, k_out, v_out)`` with v, as ``[B * heads, N, d]``: what ``project``, ``attention`` and
    ``fused`` take.  ``q_weight``, ``k_weight`` ``[d]``: weights of the root-mean-square norm (None:
    no norm).  ``cos``, ``sin`` ``[rows, rotary_dim / 2]`` fp32 (None: no rotation), row ``positions[b, n]``
    (int32) or ``n``; pairs ``(i, i + rotary_dim / 2)``, or ``(2i, 2i + 1)`` if ``interleaved``."""
    B, N, hq, hk, d, rot, rows, wcode = _qk_common(q, k, v, q_weight, k_weight, cos, sin, positions)
    kv = (B, N, hk, d)
    hqs, hks, hvs = _heads(q, q.shape, "q"), _heads(k, kv, "k"), _heads(v, kv, "v")
    dt, dev = q.dtype, q.device
    q_out = torch.empty((B * hq, N, d), dtype=dt, device=dev)
    k_out = torch.empty((B * hk, N, d), dtype=dt, device=dev)
    v_out = None if v is None else torch.empty((B * hk, N, d), dtype=dt, device=dev)
    _check(api.load_library().dera_qk_norm_rope(
        hqs, hks, hvs, _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(positions), q_out.data_ptr(),
        k_out.data_ptr(), _ptr(v_out), B, N, hq, hk, d, rot, rows, interleaved, eps, _dtype(dt), wcode,
        _launch_stream(dev, stream)))
    return (q_out, k_out) if v is None else (q_out, k_out, v_out)


def qk_norm_rope_backward_workspace_size(B: int, N: int, q_heads: int, kv_heads: int, head_dim: int = 64) -> int:
    """Scratch bytes of :func:`qk_norm_rope_backward` on the current device."""
    return _size("dera_qk_norm_rope_backward_workspace_size", B, N, q_heads, kv_heads, head_dim)


def qk_norm_rope_backward(q: torch.Tensor, k: torch.Tensor, dq_out: torch.Tensor, dk_out: torch.Tensor,
                          dv_out: torch.Tensor | None = None, *, q_weight: torch.Tensor | None = None,
                          k_weight: torch.Tensor | None = None, cos: torch.Tensor | None = None,
                          sin: torch.Tensor | None = None, positions: torch.Tensor | None = None, eps: float = 1e-6,
                          interleaved: bool = False, grad_dtype: torch.dtype | None = None,
                          dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                          dv: torch.Tensor | None = None, stream=None, workspace: torch.Tensor | None = None):
    """Gradients of :func:`qk_norm_rope` via ``dera_qk_norm_rope_backward``:
    ``(dq, dk, dv, dq_weight, dk_weight)``.

    q and k are the forward's; ``dq_out``, ``dk_out``, ``dv_out`` the gradients of its outputs, fp32 or
    of q's dtype.  dq, dk and dv (None without ``dv_out``) come back in token order in ``grad_dtype``
    (default fp32), or are written to the tensors given, which may be slices of one packed
    gradient; the weights' gradients are fp32 (None without weights)."""
    B, N, hq, hk, d, rot, rows, wcode = _qk_common(q, k, None, q_weight, k_weight, cos, sin, positions)
    norm = q_weight is not None
    given = [t for t in (dq, dk, dv) if t is not None]
    gd = grad_dtype or (given[0].dtype if given else torch.float32)
    if any(t.dtype != gd for t in given):
        raise TypeError(f"dq, dk and dv must be {gd}")
    if dv is not None and dv_out is None:
        raise ValueError("dv needs dv_out")
    if dk_out.dtype != dq_out.dtype or (dv_out is not None and dv_out.dtype != dq_out.dtype):
        raise TypeError("dq_out, dk_out and dv_out must share a dtype")
    _want(dq_out, (B * hq, N, d), "dq_out")
    _want(dk_out, (B * hk, N, d), "dk_out")
    if dv_out is not None:
        _want(dv_out, (B * hk, N, d), "dv_out")
    dev = q.device
    dq = torch.empty((B, N, hq, d), dtype=gd, device=dev) if dq is None else dq
    dk = torch.empty((B, N, hk, d), dtype=gd, device=dev) if dk is None else dk
    if dv is None and dv_out is not None:
        dv = torch.empty((B, N, hk, d), dtype=gd, device=dev)
    kv = (B, N, hk, d)
    hqs, hks = _heads(q, q.shape, "q"), _heads(k, kv, "k")
    hdq, hdk, hdv = _heads(dq, q.shape, "dq"), _heads(dk, kv, "dk"), _heads(dv, kv, "dv")
    dqw = _like(q_weight, torch.float32) if norm else None
    dkw = _like(k_weight, torch.float32) if norm else None
    st = _launch_stream(dev, stream)
    keep, ws, ws_bytes = None, None, 0
    if norm:
        keep, ws, ws_bytes = _scratch(dev, stream, st, workspace, "dera_qk_norm_rope_backward_workspace_size", B, N, hq,
                                      hk, d)
    _check(api.load_library().dera_qk_norm_rope_backward(
        hqs, hks, _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(positions), dq_out.data_ptr(),
        dk_out.data_ptr(), _ptr(dv_out), hdq, hdk, hdv, _ptr(dqw), _ptr(dkw), B, N, hq, hk, d, rot, rows, interleaved,
        eps, _dtype(q.dtype), wcode, _dtype(dq_out.dtype), _dtype(gd), ws, ws_bytes, st))
    return dq, dk, dv, dqw, dkw


# ------------------------------------------------------------------------------------- attention
def attention_lse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rel_h: torch.Tensor, rel_w: torch.Tensor,
                  H: int, W: int, scale: float | None = None, out_dtype: torch.dtype | None = None, stream=None,
                  workspace=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Training forward of the two-step form via ``dera_relpos_attention_lse``: ``(out, lse)``, lse
    ``[BH, N]`` fp32 (base 2).  A bias of -inf masks its keys; a row with every key masked gives
    out = 0 and lse = -inf.  ``workspace``: a caller-owned uint8 tensor that no other call in flight
    uses, None for a buffer of this call, or False for none (whole units)."""
    BH, N, d = q.shape
    _fits(BH | H | W | d)
    scale = d ** -0.5 if scale is None else scale
    size = (BH, H * W, d)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _want(t, size, name)
    _want(rel_h, (BH, N, H), "rel_h")
    _want(rel_w, (BH, N, W), "rel_w")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share a dtype")
    if rel_h.dtype != rel_w.dtype:
        raise TypeError("rel_h and rel_w must share a dtype")
    out = _like(q, out_dtype or q.dtype)
    lse = torch.empty((BH, N), dtype=torch.float32, device=q.device)
    st = _launch_stream(q.device, stream)
    # a buffer of this call, not the stream's: graphs captured on one stream may be replayed side by side
    keep, ws, ws_bytes = ((None, None, 0) if workspace is False else
                          _scratch(q.device, stream, st, workspace, "dera_relpos_workspace_size", BH, H, W, d))
    _check(api.load_library().dera_relpos_attention_lse(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), rel_h.data_ptr(), rel_w.data_ptr(), out.data_ptr(), lse.data_ptr(),
        BH, H, W, d, scale, _dtype(q.dtype), _dtype(rel_h.dtype), _dtype(out.dtype), ws, ws_bytes, st))
    return out, lse


def attention_backward_workspace_size(BH: int, H: int, W: int, head_dim: int = 64) -> int:
    """Scratch bytes of :func:`attention_backward` for this size on the current device."""
    return _size("dera_relpos_attention_backward_workspace_size", BH, H, W, head_dim)


def attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rel_h: torch.Tensor, rel_w: torch.Tensor,
                       out: torch.Tensor, lse: torch.Tensor, dout: torch.Tensor, H: int, W: int,
                       scale: float | None = None, grad_dtype: torch.dtype | None = None, stream=None,
                       workspace: torch.Tensor | None = None):
    """Gradients of :func:`attention_lse` via ``dera_relpos_attention_backward``:
    ``(dq, dk, dv, drel_h, drel_w)``; dq, dk, dv in ``grad_dtype`` (default fp32), the bias's fp32
    (exactly zero along an axis of length one).
    ``out`` and ``lse`` come from :func:`attention_lse`.  ``workspace``: a caller-owned uint8 tensor that
    no other call in flight uses, or None for a buffer of this call."""
    BH, N, d = q.shape
    _fits(BH | H | W | d)
    scale = d ** -0.5 if scale is None else scale
    gd = grad_dtype or torch.float32
    size, size_h, size_w = (BH, H * W, d), (BH, N, H), (BH, N, W)
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _want(t, size, name)
    _want(lse, (BH, N), "lse")
    _want(rel_h, size_h, "rel_h")
    _want(rel_w, size_w, "rel_w")
    if k.dtype != q.dtype or v.dtype != q.dtype or dout.dtype != q.dtype:
        raise TypeError("q, k, v and dout must share a dtype")
    if rel_h.dtype != rel_w.dtype:
        raise TypeError("rel_h and rel_w must share a dtype")
    if lse.dtype != torch.float32:
        raise TypeError("lse must be float32")
    dev = q.device
    dq, dk, dv = _like(q, gd), _like(k, gd), _like(v, gd)
    drel_h, drel_w = _like(rel_h, torch.float32), _like(rel_w, torch.float32)
    st = _launch_stream(dev, stream)
    keep, ws, ws_bytes = _scratch(dev, stream, st, workspace, "dera_relpos_attention_backward_workspace_size", BH, H, W, d)
    _check(api.load_library().dera_relpos_attention_backward(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), rel_h.data_ptr(), rel_w.data_ptr(), out.data_ptr(), lse.data_ptr(),
        dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), drel_h.data_ptr(), drel_w.data_ptr(), BH, H, W, d,
        scale, _dtype(q.dtype), _dtype(rel_h.dtype), _dtype(out.dtype), _dtype(gd), ws, ws_bytes, st))
    return dq, dk, dv, drel_h, drel_w


# ------------------------------------------------------------------------------------ projection
def project_backward_workspace_size(BH: int, H: int, W: int, head_dim: int = 64) -> int:
    """Scratch bytes of :func:`project_backward` for this size on the current device."""
    return _size("dera_relpos_project_backward_workspace_size", BH, H, W, head_dim)


def project_backward(q: torch.Tensor, rel_pos_h: torch.Tensor, rel_pos_w: torch.Tensor, drel_h: torch.Tensor,
                     drel_w: torch.Tensor, H: int, W: int, dq: torch.Tensor | None = None,
                     grad_dtype: torch.dtype | None = None, stream=None, workspace: torch.Tensor | None = None):
    """Gradients of :func:`~relative_position_bias_gb300.project` via ``dera_relpos_project_backward``:
    ``(dq, drel_pos_h, drel_pos_w)``.

    ``drel_h``, ``drel_w``: the compact bias's gradient, fp32.  ``dq``, if given, is the attention's part
    of dq, to which the projection's is added (in a new tensor of the same dtype); else dq comes in
    ``grad_dtype`` (default fp32).  The tables' gradients are fp32."""
    BH, N, d = q.shape
    _fits(BH | H | W | d)
    gd = grad_dtype or (torch.float32 if dq is None else dq.dtype)
    size, size_h, size_w = (BH, H * W, d), (2 * H - 1, d), (2 * W - 1, d)
    _want(q, size, "q")
    _want(rel_pos_h, size_h, "rel_pos_h")
    _want(rel_pos_w, size_w, "rel_pos_w")
    if rel_pos_h.dtype != q.dtype or rel_pos_w.dtype != q.dtype:
        raise TypeError("q and the tables must share a dtype")
    _same(drel_h, (BH, N, H), torch.float32, "drel_h")
    _same(drel_w, (BH, N, W), torch.float32, "drel_w")
    _same(dq, (BH, N, d), gd, "dq")
    dev = q.device
    out, dth, dtw = _like(q, gd), _like(rel_pos_h, torch.float32), _like(rel_pos_w, torch.float32)
    st = _launch_stream(dev, stream)
    keep, ws, ws_bytes = _scratch(dev, stream, st, workspace, "dera_relpos_project_backward_workspace_size", BH, H, W, d)
    _check(api.load_library().dera_relpos_project_backward(
        q.data_ptr(), rel_pos_h.data_ptr(), rel_pos_w.data_ptr(), drel_h.data_ptr(), drel_w.data_ptr(), _ptr(dq),
        out.data_ptr(), dth.data_ptr(), dtw.data_ptr(), BH, H, W, d, _dtype(q.dtype), _dtype(gd), ws, ws_bytes, st))
    return out, dth, dtw
