"""The entry points of include/dera_block.h without a GPU: declared, exported, and every bad argument
refused on the host before any CUDA work."""
from __future__ import annotations

import ctypes
import subprocess

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import api, block
from relative_position_bias_gb300 import build as rbuild

CODES = {n: c for c, n in api.STATUS_NAMES.items()}
FAKE = 0x10000          # aligned, never dereferenced
FAKE_MISALIGNED = 0x10008
F16, BF16, F32 = 0, 1, 2
PAST = (CODES["DERA_ERR_CUDA"], CODES["DERA_ERR_DEVICE"])   # argument checks passed; no device (or no such memory)


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rpb.load_library()


class Heads(ctypes.Structure):
    """``dera_heads``"""
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_longlong), ("stride_token", ctypes.c_longlong),
                ("stride_head", ctypes.c_longlong)]


def _at(h):
    return None if h is None else ctypes.byref(h)


def test_header_and_exports(lib):
    names = set(rpb.declared_entry_points(block.HEADER))
    assert names == {"dera_layer_norm", "dera_layer_norm_backward", "dera_layer_norm_backward_workspace_size",
                     "dera_linear", "dera_linear_backward",
                     "dera_linear_backward_workspace_size", "dera_activation_backward"}
    out = subprocess.run(["nm", "-D", "--defined-only", rbuild.LIB], capture_output=True, text=True, check=True)
    exported = {line.split()[-1] for line in out.stdout.splitlines() if " T " in line}
    assert names <= exported
    assert not {s for s in exported if s.startswith("_ZN4dera")}
    with open(block.HEADER) as fh:
        text = fh.read()
    for name, code in block.ACTIVATIONS.items():
        assert f"DERA_ACT_{(name or 'none').upper()} = {code}" in text


# ------------------------------------------------------------------------------------- layer norm
def _ln(lib, *, ptrs=(FAKE,) * 6, rows=3, cols=64, xs=64, eps=1e-6, in_dt=BF16, w_dt=F32, out_dt=BF16):
    return lib.dera_layer_norm(*ptrs, rows, cols, xs, eps, in_dt, w_dt, out_dt, None)


def _ln_bwd(lib, *, ptrs=(FAKE,) * 9, rows=3, cols=64, xs=64, in_dt=BF16, w_dt=F32, z_dt=BF16, g_dt=BF16, ws=FAKE):
    return lib.dera_layer_norm_backward(*ptrs, rows, cols, xs, in_dt, w_dt, z_dt, g_dt, ws, 1 << 30, None)


@pytest.mark.parametrize("call", [_ln, _ln_bwd])
def test_layer_norm_refusals(lib, call):
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=16385), dict(xs=63)):
        assert call(lib, **bad) == CODES["DERA_ERR_SHAPE"], bad
    for bad in (dict(in_dt=3), dict(w_dt=F16), dict(w_dt=7)):
        assert call(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    other = dict(out_dt=F16) if call is _ln else dict(z_dt=F16)
    assert call(lib, **other) == CODES["DERA_ERR_DTYPE"]
    assert call(lib, rows=1, xs=0) in PAST                     # the stride of a single row is not looked at
    n = 6 if call is _ln else 9
    optional = {1, 2} if call is _ln else {4, 5}               # weight and bias; weight and dres
    for i in range(n):
        ptrs = [FAKE] * n
        ptrs[i] = None
        want = PAST if i in optional and not (call is _ln and i == 1) else (CODES["DERA_ERR_NULL"],)
        assert call(lib, ptrs=tuple(ptrs)) in want, i
        ptrs[i] = FAKE + 1                                     # off its elements
        assert call(lib, ptrs=tuple(ptrs)) in (CODES["DERA_ERR_ALIGN"], CODES["DERA_ERR_CUDA"]), i
    assert call(lib, rows=0, ptrs=(None,) * n) == 0
    if call is _ln:
        for eps in (-1.0, float("nan"), float("inf")):
            assert call(lib, eps=eps) == CODES["DERA_ERR_SHAPE"]


def test_layer_norm_sizes(lib):
    n = ctypes.c_size_t(7)
    size = lib.dera_layer_norm_backward_workspace_size
    assert size(1, 4, None) == CODES["DERA_ERR_NULL"]
    assert size(-1, 4, ctypes.byref(n)) == size(1, 0, ctypes.byref(n)) == CODES["DERA_ERR_SHAPE"]
    assert size(0, 4, ctypes.byref(n)) == 0 and n.value == 0


def test_layer_norm_binding_checks():
    x, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.ones(8)
    m = torch.zeros(3)
    for bad in ((x, w[:4]), (x, None, w), (x, w, w[:4]), (x.t(), torch.ones(3)), (torch.zeros(()), None)):
        with pytest.raises(ValueError):
            rpb.layer_norm(*bad)
    for bad in ((x, w.double()), (x, w.half()), (x, w, w.bfloat16()), (x.double(), None)):
        with pytest.raises(TypeError):
            rpb.layer_norm(*bad)
    with pytest.raises(rpb.DeraError) as e:
        rpb.layer_norm(x, w, out_dtype=torch.float16)
    assert e.value.status == CODES["DERA_ERR_DTYPE"]
    for bad in ((x[:2], x, m, m, w), (x, x, m[:2], m, w), (x, x, m, m, w[:2])):
        with pytest.raises(ValueError):
            rpb.layer_norm_backward(*bad)
    with pytest.raises(TypeError):
        rpb.layer_norm_backward(x, x, m.double(), m, w)
    with pytest.raises(TypeError):
        rpb.layer_norm_backward(x, x, m, m, w, dres=x, grad_dtype=torch.float32)
    with pytest.raises(rpb.DeraError) as e:                    # CPU tensors are not device memory
        rpb.layer_norm(x, w)
    assert e.value.status in PAST


# ----------------------------------------------------------------------------------------- linear
def _x(p=FAKE, sb=64 * 12, st=64, sh=64):
    return Heads(p, sb, st, sh)


def _lin(lib, *, x=None, w=FAKE, b=FAKE, res=FAKE, y=FAKE, pre=FAKE, B=2, N=3, heads=1, d=64, out=72, act=2, in_dt=BF16,
         b_dt=F32, out_dt=BF16):
    return lib.dera_linear(_at(x or _x()), w, b, res, y, pre, B, N, heads, d, out, act, in_dt, b_dt, out_dt, None)


def _lin_bwd(lib, *, dy=FAKE, x=None, w=FAKE, ip=None, dx=None, dw=FAKE, db=FAKE, B=2, N=3, heads=1, d=64, out=72, act=0,
             in_dt=BF16, g_dt=F32, w_dt=F32, no_dx=False):
    return lib.dera_linear_backward(dy, _at(x or _x()), w, _at(ip), None if no_dx else _at(dx or _x()), dw, db, B, N, heads,
                                    d, out, act, in_dt, g_dt, w_dt, FAKE, 1 << 40, None)


@pytest.mark.parametrize("call", [_lin, _lin_bwd])
def test_linear_refusals(lib, call):
    for bad in (dict(B=-1), dict(N=-1), dict(heads=0), dict(d=0), dict(out=0), dict(d=60), dict(out=70),
                dict(heads=3, d=72), dict(B=1 << 16, N=1 << 16), dict(d=(1 << 20) + 8), dict(heads=1 << 15, d=64),
                dict(out=(1 << 20) + 8)):
        assert call(lib, **bad) == CODES["DERA_ERR_SHAPE"], bad
    for bad in (dict(in_dt=F32), dict(act=6), dict(act=-1)):
        assert call(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    for bad in (dict(x=Heads(None, 0, 0, 0)), dict(w=None)):
        assert call(lib, **bad) == CODES["DERA_ERR_NULL"], bad
    for bad in (dict(x=_x(FAKE_MISALIGNED)), dict(x=_x(st=60)), dict(w=FAKE_MISALIGNED)):
        assert call(lib, **bad) == CODES["DERA_ERR_ALIGN"], bad
    for bad in (dict(x=_x(st=-64)), dict(x=_x(st=0)), dict(x=_x(sb=0)), dict(x=_x(sb=1 << 37))):
        assert call(lib, **bad) == CODES["DERA_ERR_SHAPE"], bad
    assert call(lib, B=1, N=1, x=_x(sb=0, st=0, sh=0)) in PAST
    more = {} if call is _lin else dict(dx=_x(st=128, sh=64))
    assert call(lib, heads=2, x=_x(st=128, sh=64), **more) in PAST


def test_linear_refuses_the_rest(lib):
    assert _lin(lib, y=None) == CODES["DERA_ERR_NULL"]
    for name in ("b", "res", "y", "pre"):
        assert _lin(lib, **{name: FAKE_MISALIGNED}) == CODES["DERA_ERR_ALIGN"], name
    for bad in (dict(b_dt=F16), dict(out_dt=F16)):
        assert _lin(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    assert _lin(lib, b=None, b_dt=9, res=None, pre=None, act=0) in PAST
    assert _lin(lib, B=0, w=None, y=None) == _lin(lib, N=0, x=Heads(None, 0, 0, 0)) == 0
    assert _lin_bwd(lib, dy=None) == CODES["DERA_ERR_NULL"]
    assert _lin_bwd(lib, act=2) == CODES["DERA_ERR_NULL"]                 # an activation without what it was given
    assert _lin_bwd(lib, ip=_x()) == CODES["DERA_ERR_NULL"]               # and the other way round
    for name in ("dy", "dw", "db"):
        assert _lin_bwd(lib, **{name: FAKE_MISALIGNED}) == CODES["DERA_ERR_ALIGN"], name
    for bad in (dict(g_dt=F16), dict(w_dt=F16)):
        assert _lin_bwd(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    assert _lin_bwd(lib, dx=_x(st=8)) == CODES["DERA_ERR_SHAPE"]          # rows of the gradient that share elements
    # what is not asked for needs nothing
    assert _lin_bwd(lib, no_dx=True, w=None) in PAST
    assert _lin_bwd(lib, dw=None, x=Heads(None, 0, 0, 0)) in PAST
    assert _lin_bwd(lib, B=0, dw=None, db=None, dy=None) == 0


def test_linear_sizes(lib):
    n = ctypes.c_size_t(7)
    size = lib.dera_linear_backward_workspace_size
    assert size(1, 1, 1, 8, 8, None) == CODES["DERA_ERR_NULL"]
    assert size(1, 1, 1, 8, 7, ctypes.byref(n)) == CODES["DERA_ERR_SHAPE"]
    assert size(0, 5, 1, 8, 8, ctypes.byref(n)) == 0 and n.value == 0


def test_linear_binding_checks():
    x, w, b = torch.zeros(2, 3, 64).bfloat16(), torch.zeros(72, 64).bfloat16(), torch.zeros(72)
    dy = torch.zeros(2, 3, 72).bfloat16()
    for bad in (dict(bias=b[:8]), dict(residual=x), dict(activation="tanh")):
        with pytest.raises(ValueError):
            rpb.linear(x, w, **bad)
    for args in ((x[..., :56], w), (x, w[0]), (x[None, None], w), (torch.zeros(2, 3, 2, 64).bfloat16(), w),
                 (x.transpose(1, 2), torch.zeros(72, 3).bfloat16())):
        with pytest.raises(ValueError):
            rpb.linear(*args)
    for bad in (dict(bias=b.half()), dict(residual=dy.float())):
        with pytest.raises(TypeError):
            rpb.linear(x, w, **bad)
    with pytest.raises(TypeError):
        rpb.linear(x, w.half())
    with pytest.raises(ValueError):
        rpb.linear_backward(dy[:1], x, w)
    with pytest.raises(TypeError):
        rpb.linear_backward(dy.float(), x, w)
    for bad in (dict(input_pre=x), dict(input_activation="gelu"), dict(input_pre=x.half(), input_activation="gelu"),
                dict(input_pre=x[:1], input_activation="gelu")):
        with pytest.raises(ValueError):
            rpb.linear_backward(dy, x, w, **bad)
    with pytest.raises(rpb.DeraError) as e:
        rpb.linear(x, w)
    assert e.value.status in PAST


# ------------------------------------------------------------------------------------- activation
def test_activation_backward_refusals(lib):
    def call(ptrs=(FAKE,) * 3, n=8, act=2, p_dt=BF16, z_dt=BF16, g_dt=F32):
        return lib.dera_activation_backward(*ptrs, n, act, p_dt, z_dt, g_dt, None)

    assert call(n=-1) == CODES["DERA_ERR_SHAPE"]
    for bad in (dict(act=0), dict(act=6), dict(p_dt=4), dict(z_dt=F16), dict(g_dt=F16)):
        assert call(**bad) == CODES["DERA_ERR_DTYPE"], bad
    for i in range(3):
        ptrs = [FAKE] * 3
        ptrs[i] = None
        assert call(tuple(ptrs)) == CODES["DERA_ERR_NULL"]
        ptrs[i] = FAKE_MISALIGNED
        assert call(tuple(ptrs)) == CODES["DERA_ERR_ALIGN"]
    assert call((None,) * 3, n=0) == 0
    x = torch.zeros(8)
    for act in (None, "elu"):
        with pytest.raises(ValueError):
            rpb.activation_backward(x, x, act)
    with pytest.raises(ValueError):
        rpb.activation_backward(x[:4], x, "gelu")
