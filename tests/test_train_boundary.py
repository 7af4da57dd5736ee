"""The entry points of include/dera_train.h without a GPU: declared, exported, and every bad argument
refused on the host before any CUDA work."""
from __future__ import annotations

import ctypes
import subprocess

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import api, train
from relative_position_bias_gb300 import build as rbuild

CODES = {n: c for c, n in api.STATUS_NAMES.items()}
FAKE = 0x10000          # aligned, never dereferenced
FAKE_MISALIGNED = 0x10008
F16, BF16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rpb.load_library()


def test_header_and_exports(lib):
    names = set(rpb.declared_entry_points(train.HEADER))
    assert names == {"dera_qk_norm_rope", "dera_qk_norm_rope_backward", "dera_qk_norm_rope_backward_workspace_size",
                     "dera_relpos_attention_lse", "dera_relpos_attention_backward",
                     "dera_relpos_attention_backward_workspace_size", "dera_relpos_project_backward",
                     "dera_relpos_project_backward_workspace_size"}
    out = subprocess.run(["nm", "-D", "--defined-only", rbuild.LIB], capture_output=True, text=True, check=True)
    exported = {line.split()[-1] for line in out.stdout.splitlines() if " T " in line}
    assert names <= exported
    assert not {s for s in exported if s.startswith("_ZN4dera")}


# ------------------------------------------------------------------------------ norms and rotation
class Heads(ctypes.Structure):
    """``dera_heads``"""
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_longlong), ("stride_token", ctypes.c_longlong),
                ("stride_head", ctypes.c_longlong)]


def _h(p=FAKE, sb=64 * 12, st=64 * 4, sh=64):
    return Heads(p, sb, st, sh)


def _at(h):
    return None if h is None else ctypes.byref(h)


def _qk(lib, *, q=None, k=None, v=None, qw=FAKE, kw=FAKE, cos=FAKE, sin=FAKE, pos=None, qo=FAKE, ko=FAKE, vo=None, B=2,
        N=3, hq=2, hk=1, d=64, rot=64, rows=3, eps=1e-6, in_dt=BF16, w_dt=BF16):
    return lib.dera_qk_norm_rope(_at(q or _h()), _at(k or _h()), _at(v), qw, kw, cos, sin, pos, qo, ko, vo, B, N, hq, hk,
                                 d, rot, rows, 0, eps, in_dt, w_dt, None)


def _qk_bwd(lib, *, q=None, k=None, qw=FAKE, kw=FAKE, cos=FAKE, sin=FAKE, pos=None, zq=FAKE, zk=FAKE, zv=None, dq=None,
            dk=None, dv=None, dqw=FAKE, dkw=FAKE, B=2, N=3, hq=2, hk=1, d=64, rot=64, rows=3, eps=1e-6, in_dt=BF16,
            w_dt=BF16, z_dt=BF16, g_dt=F32):
    return lib.dera_qk_norm_rope_backward(_at(q or _h()), _at(k or _h()), qw, kw, cos, sin, pos, zq, zk, zv,
                                          _at(dq or _h()), _at(dk or _h()), _at(dv), dqw, dkw, B, N, hq, hk, d, rot,
                                          rows, 0, eps, in_dt, w_dt, z_dt, g_dt, FAKE, 1 << 30, None)


@pytest.mark.parametrize("call", [_qk, _qk_bwd])
def test_qk_norm_rope_refusals(lib, call):
    assert call(lib, d=32) == CODES["DERA_ERR_HEAD_DIM"]
    for bad in (dict(B=-1), dict(N=-1), dict(hq=0), dict(hk=0), dict(hq=16385), dict(B=1 << 16, N=1 << 16),
                dict(rot=8), dict(rot=80), dict(rot=-16), dict(rows=2), dict(rows=0, pos=FAKE), dict(eps=-1e-6),
                dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(lib, **bad) == CODES["DERA_ERR_SHAPE"], bad
    for bad in (dict(in_dt=F32), dict(w_dt=F16), dict(w_dt=7)):
        assert call(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    for bad in (dict(qw=None), dict(kw=None), dict(q=Heads(None, 0, 0, 0)), dict(v=_h()) if call is _qk else dict(dv=_h())):
        assert call(lib, **bad) == CODES["DERA_ERR_NULL"], bad
    for bad in (dict(q=_h(FAKE_MISALIGNED)), dict(k=_h(st=64 * 4 + 4)), dict(q=_h(sh=60))):
        assert call(lib, **bad) == CODES["DERA_ERR_ALIGN"], bad
    assert call(lib, q=_h(st=-256)) == CODES["DERA_ERR_SHAPE"]
    # an empty batch: no CUDA call, and without weights no pointer is looked at
    assert call(lib, B=0, qw=None, kw=None, cos=None, sin=None, q=Heads(None, 0, 0, 0)) == 0
    assert call(lib, N=0, rows=0, rot=0, qw=None, kw=None) == 0


def test_qk_norm_rope_refuses_the_rest(lib):
    assert _qk(lib, qo=None) == CODES["DERA_ERR_NULL"]
    assert _qk(lib, ko=FAKE_MISALIGNED) == CODES["DERA_ERR_ALIGN"]
    assert _qk_bwd(lib, zq=None) == CODES["DERA_ERR_NULL"]
    assert _qk_bwd(lib, dqw=None) == CODES["DERA_ERR_NULL"]
    assert _qk_bwd(lib, z_dt=F16) == CODES["DERA_ERR_DTYPE"]
    assert _qk_bwd(lib, g_dt=F16) == CODES["DERA_ERR_DTYPE"]
    # rows of an output that share elements: a repeated head, tokens closer than the heads they hold
    assert _qk_bwd(lib, dq=_h(sh=0)) == CODES["DERA_ERR_SHAPE"]
    assert _qk_bwd(lib, dq=_h(st=64)) == CODES["DERA_ERR_SHAPE"]
    assert _qk_bwd(lib, dk=_h(sb=64 * 4)) == CODES["DERA_ERR_SHAPE"]
    # ... while rows that only interleave (one head of 64 every 256, the next batch 128 further), and
    # an order of dimensions other than batch, token, head, are fine as far as the host can see
    for fine in (dict(dk=_h(sb=64 * 2)), dict(dq=_h(sb=64 * 3 * 2, st=64, sh=64 * 3))):
        assert _qk_bwd(lib, **fine) in (CODES["DERA_ERR_CUDA"], CODES["DERA_ERR_DEVICE"])


def test_qk_binding_checks():
    q, k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    w, c = torch.ones(64, dtype=torch.bfloat16), torch.zeros(3, 32)
    for bad in (dict(q_weight=w), dict(cos=c), dict(positions=torch.zeros(2, 3, dtype=torch.int32)),
                dict(q_weight=w[:32], k_weight=w[:32]), dict(cos=c, sin=c[:2])):
        with pytest.raises(ValueError):
            rpb.qk_norm_rope(q, k, **bad)
    with pytest.raises(ValueError):
        rpb.qk_norm_rope(q, k[:, :2])
    with pytest.raises(ValueError):
        rpb.qk_norm_rope(q.transpose(2, 3), k)
    for bad in (dict(q_weight=w.half(), k_weight=w.half()), dict(cos=c.half(), sin=c.half()),
                dict(cos=c, sin=c, positions=torch.zeros(2, 3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            rpb.qk_norm_rope(q, k, **bad)
    with pytest.raises(TypeError):
        rpb.qk_norm_rope(q, k.half())
    zq, zk = torch.zeros(8, 3, 64, dtype=torch.bfloat16), torch.zeros(4, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rpb.qk_norm_rope_backward(q, k, zq, zk, dv=k)          # dv without dv_out
    with pytest.raises(TypeError):
        rpb.qk_norm_rope_backward(q, k, zq, zk.float())
    with pytest.raises(TypeError):
        rpb.qk_norm_rope_backward(q, k, zq, zk, dq=q, grad_dtype=torch.float32)
    with pytest.raises(rpb.DeraError) as e:                    # CPU tensors are not device memory
        rpb.qk_norm_rope(q, k)
    assert e.value.status in (6, 8)


# ------------------------------------------------------------------------------------- attention
def _lse(lib, *, ptrs=(FAKE,) * 7, BH=1, H=4, W=4, d=64, in_dt=BF16, bias_dt=F32, out_dt=F32):
    return lib.dera_relpos_attention_lse(*ptrs, BH, H, W, d, 0.125, in_dt, bias_dt, out_dt, None, 0, None)


def test_attention_lse_refusals(lib):
    assert _lse(lib, d=32) == CODES["DERA_ERR_HEAD_DIM"]
    assert _lse(lib, H=65) == CODES["DERA_ERR_SHAPE"]
    assert _lse(lib, in_dt=F32) == CODES["DERA_ERR_DTYPE"]
    assert _lse(lib, bias_dt=4) == CODES["DERA_ERR_DTYPE"]
    assert _lse(lib, out_dt=F16) == CODES["DERA_ERR_DTYPE"]
    for i in range(7):
        ptrs = [FAKE] * 7
        ptrs[i] = None
        assert _lse(lib, ptrs=tuple(ptrs)) == CODES["DERA_ERR_NULL"]
        ptrs[i] = FAKE_MISALIGNED
        assert _lse(lib, ptrs=tuple(ptrs)) == CODES["DERA_ERR_ALIGN"]
    assert _lse(lib, BH=0, ptrs=(None,) * 7) == 0


def _bwd(lib, *, ptrs=(FAKE,) * 13, BH=1, H=4, W=4, d=64, in_dt=BF16, bias_dt=F32, out_dt=F32, grad_dt=F32):
    return lib.dera_relpos_attention_backward(*ptrs, BH, H, W, d, 0.125, in_dt, bias_dt, out_dt, grad_dt, FAKE, 1 << 30,
                                              None)


def test_attention_backward_refusals(lib):
    assert _bwd(lib, d=32) == CODES["DERA_ERR_HEAD_DIM"]
    for bad in (dict(H=0), dict(W=65), dict(BH=-1), dict(BH=1 << 26, H=64, W=64)):
        assert _bwd(lib, **bad) == CODES["DERA_ERR_SHAPE"], bad
    for bad in (dict(in_dt=F32), dict(bias_dt=3), dict(out_dt=F16), dict(grad_dt=F16)):
        assert _bwd(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    for i in range(13):
        ptrs = [FAKE] * 13
        ptrs[i] = None
        assert _bwd(lib, ptrs=tuple(ptrs)) == CODES["DERA_ERR_NULL"]
        ptrs[i] = FAKE_MISALIGNED
        assert _bwd(lib, ptrs=tuple(ptrs)) == CODES["DERA_ERR_ALIGN"]
    assert _bwd(lib, BH=0, ptrs=(None,) * 13) == 0
    n = ctypes.c_size_t(7)
    size = lib.dera_relpos_attention_backward_workspace_size
    assert size(1, 4, 4, 64, None) == CODES["DERA_ERR_NULL"]
    assert size(1, 4, 4, 32, ctypes.byref(n)) == CODES["DERA_ERR_HEAD_DIM"]
    assert size(0, 4, 4, 64, ctypes.byref(n)) == 0 and n.value == 0


def test_attention_binding_checks():
    q = torch.zeros(2, 6, 64, dtype=torch.bfloat16)
    rh, rw, lse = torch.zeros(2, 6, 2), torch.zeros(2, 6, 3), torch.zeros(2, 6)
    with pytest.raises(ValueError):
        rpb.attention_lse(q, q, q, rw, rh, 2, 3)
    with pytest.raises(TypeError):
        rpb.attention_lse(q, q, q, rh, rw.half(), 2, 3)
    with pytest.raises(TypeError):
        rpb.attention_backward(q, q, q, rh, rw, q, lse.double(), q, 2, 3)
    with pytest.raises(TypeError):
        rpb.attention_backward(q, q, q, rh, rw, q, lse, q.float(), 2, 3)
    with pytest.raises(ValueError):
        rpb.attention_backward(q, q, q, rh, rw, q, lse[:1], q, 2, 3)


def _pb(lib, *, ptrs=(FAKE,) * 5 + (None,) + (FAKE,) * 3, BH=1, H=4, W=4, d=64, in_dt=BF16, grad_dt=F32):
    return lib.dera_relpos_project_backward(*ptrs, BH, H, W, d, in_dt, grad_dt, FAKE, 1 << 30, None)


def test_project_backward_refusals(lib):
    assert _pb(lib, d=96) == CODES["DERA_ERR_HEAD_DIM"]
    for bad in (dict(H=65), dict(W=0), dict(BH=-1)):
        assert _pb(lib, **bad) == CODES["DERA_ERR_SHAPE"], bad
    for bad in (dict(in_dt=F32), dict(grad_dt=F16)):
        assert _pb(lib, **bad) == CODES["DERA_ERR_DTYPE"], bad
    for i in range(9):
        ptrs = [FAKE] * 9
        ptrs[i] = None
        if i != 5:    # dq_in is optional
            assert _pb(lib, ptrs=tuple(ptrs)) == CODES["DERA_ERR_NULL"]
        ptrs[i] = FAKE_MISALIGNED
        assert _pb(lib, ptrs=tuple(ptrs)) == CODES["DERA_ERR_ALIGN"]
    assert _pb(lib, BH=0, ptrs=(None,) * 9) == CODES["DERA_ERR_NULL"]    # the tables' gradients are still written


def test_project_backward_binding_checks():
    q, th, tw = torch.zeros(2, 6, 64).half(), torch.zeros(3, 64).half(), torch.zeros(5, 64).half()
    gh, gw = torch.zeros(2, 6, 2), torch.zeros(2, 6, 3)
    with pytest.raises(ValueError):
        rpb.project_backward(q, tw, th, gh, gw, 2, 3)
    with pytest.raises(TypeError):
        rpb.project_backward(q, th, tw, gh.half(), gw.half(), 2, 3)
    with pytest.raises(TypeError):
        rpb.project_backward(q, th, tw, gh, gw, 2, 3, dq=q.float(), grad_dtype=torch.float16)
    with pytest.raises(TypeError):
        rpb.project_backward(q, th.float(), tw, gh, gw, 2, 3)
