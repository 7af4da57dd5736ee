"""Sizes that the C entry points' 32-bit arguments do not hold are refused, and never cut (2^32 rows to none, 2^32 + 8 columns to 8).
Tensors without memory stand for those that a device has room for."""
from __future__ import annotations

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild

BF, F32 = torch.bfloat16, torch.float32
PAST = [1 << 31, (1 << 32) - 8, 1 << 32, (1 << 32) + 8]
SHAPE = 2   # DERA_ERR_SHAPE


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


def refused(call, *args, **kw):
    with pytest.raises(rpb.DeraError) as e:
        call(*args, **kw)
    assert e.value.status == SHAPE, e.value


@pytest.mark.parametrize("n", PAST)
def test_layer_norm(n):
    for x in (m(n, 1), m(n // 8, 8, 2), m(1, n), m(0, n), m(n), m(2, n, 16)[:, :, :8]):   # rows, columns, rows at a stride
        rows = m(*x.shape[:-1], dtype=F32)
        refused(rpb.layer_norm, x)
        refused(rpb.layer_norm_backward, m(*x.shape), x, rows, rows, m(x.shape[-1], dtype=F32))
    refused(rpb.layer_norm_backward_workspace_size, n, 8)
    refused(rpb.layer_norm_backward_workspace_size, 8, n)


@pytest.mark.parametrize("n", PAST)
def test_linear(n):
    for x, out in ((m(n, 8), 8), (m(n, 1, 8), 8), (m(1, n, 8), 8), (m(n, 0, 8), 8), (m(1, n), 8), (m(n), 8), (m(3, 8), n),
                   (m(1, 1, n // 8, 8), 8), (m(1, 1, n, 1), 8), (m(n, 1, 2, 64), 8)):
        K = x.shape[2] * x.shape[3] if x.dim() == 4 else x.shape[-1]
        w = m(out, K)
        refused(rpb.linear, x, w)
        dy = m(*(x.shape[:2] if x.dim() == 4 else x.shape[:-1]), out)
        refused(rpb.linear_backward, dy, x, w)
        refused(rpb.linear_backward, dy, x, w, weight_grad=False, bias_grad=False)
    for i in range(5):
        sizes = [1, 1, 1, 8, 8]
        sizes[i] = n
        refused(rpb.linear_backward_workspace_size, *sizes)


def test_negative_sizes_are_refused_too():
    refused(rpb.linear_backward_workspace_size, -(1 << 32), 1, 1, 8, 8)
    refused(rpb.layer_norm_backward_workspace_size, -(1 << 32), 8)


@pytest.mark.parametrize("n", PAST)
def test_attention_and_projection(n):
    def grid(BH, H, W, d):
        q, lse = m(BH, H * W, d), m(BH, H * W, dtype=F32)
        th, tw, bh, bw = m(2 * H - 1, d), m(2 * W - 1, d), m(BH, H * W, H, dtype=F32), m(BH, H * W, W, dtype=F32)
        refused(rpb.project, q, th, tw, H, W)
        refused(rpb.attention, q, q, q, bh, bw, H, W, workspace=False)
        refused(rpb.attention_lse, q, q, q, bh, bw, H, W)
        refused(rpb.fused, q, q, q, th, tw, H, W)
        refused(rpb.fused_lse, q, q, q, th, tw, H, W)
        refused(rpb.fused_backward, q, q, q, th, tw, q, lse, q, H, W)
        refused(rpb.attention_backward, q, q, q, bh, bw, q, lse, q, H, W)
        refused(rpb.project_backward, q, th, tw, bh, bw, H, W)

    grid(n, 1, 1, 64)   # (a grid's sides are limited by its bias)
    grid(1, 1, 1, n)
    for i in range(4):
        sizes = [1, 1, 1, 64]
        sizes[i] = n
        for size in (rpb.workspace_size, rpb.backward_workspace_size, rpb.attention_backward_workspace_size,
                     rpb.project_backward_workspace_size):
            refused(size, *sizes)


@pytest.mark.parametrize("n", PAST)
def test_qk_norm_rope(n):
    for shape in ((n, 1, 1, 64), (1, n, 1, 64), (1, 1, n, 64), (1, 1, 1, n), (n, 0, 1, 64)):
        B, N, h, d = shape
        q, k = m(*shape), m(B, N, 1, d)
        refused(rpb.qk_norm_rope, q, k)
        refused(rpb.qk_norm_rope_backward, q, k, m(B * h, N, d), m(B, N, d))
    refused(rpb.qk_norm_rope, m(1, 1, 1, 64), m(1, 1, n, 64))
    x, table = m(1, 1, 1, 64), m(n, 1, dtype=F32)
    refused(rpb.qk_norm_rope, x, x, cos=table, sin=table)   # rows of the table
    for i in range(5):
        sizes = [1, 1, 1, 1, 64]
        sizes[i] = n
        refused(rpb.qk_norm_rope_backward_workspace_size, *sizes)
