"""How the compact-bias backward cuts its last wave of CTAs: `csrc/split.h`, compiled here and swept on the host.

The kernels take block b of a grid of `blocks(units)` as whole unit b if b < full, else as piece (b - full) % split of unit
full + (b - full) // split, whose steps are [steps p // split, steps (p + 1) // split); the workspace holds tail(units) * split
pieces."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "relative_position_bias_gb300", "csrc")
SOURCE = r"""
#include "split.h"
extern "C" void split(int units, int rs, int cs, int sms, int* out) {
  dera::CbSplit r, c;
  dera::cb_split(units, rs, cs, sms, &r, &c);
  const dera::CbSplit* both[2] = {&r, &c};
  for (int i = 0; i < 2; ++i) {
    out[4 * i] = both[i]->full;
    out[4 * i + 1] = both[i]->split;
    out[4 * i + 2] = both[i]->tail(units);
    out[4 * i + 3] = both[i]->blocks(units);
  }
}
extern "C" int rows_steps(int H, int W) { return dera::cb_rows_steps(H, W); }
extern "C" int width(int W) { return dera::cb_width(W); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("split")
    (at / "s.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(at / "s.so"),
                    str(at / "s.cpp")], check=True)
    return ctypes.CDLL(str(at / "s.so"))


def split(lib, *args):
    out = (ctypes.c_int * 8)()
    lib.split(*args, out)
    return tuple(out[:4]), tuple(out[4:])


def check(units, steps, one):
    """Every step of every unit is one block's, no block is without steps, the pieces fit the workspace."""
    full, pieces, tail, blocks = one
    assert 0 <= full <= units and pieces >= 1 and blocks == full + (units - full) * pieces
    if pieces == 1:
        assert tail == 0 and blocks == units
        return
    assert tail == units - full > 0
    assert steps // pieces >= 4
    last = 0
    for p in range(pieces):
        a, b = steps * p // pieces, steps * (p + 1) // pieces
        assert a == last and b - a >= 4
        last = b
    assert last == steps


@pytest.mark.parametrize("sms", [0, 1, 2, 16, 132, 148, 152])
def test_every_step_is_taken_once(lib, sms):
    units = sorted({u for m in range(0, 6) for d in (-2, -1, 0, 1, 2) for u in (m * sms + d, (m * sms) // 2 + d) if u > 0} | {1, 2, 3, 7, 384, 9984})
    for u in units:
        for rs, cs in ((1, 1), (4, 4), (16, 64), (64, 64), (7, 9), (40, 25), (4, 1), (32, 64), (1, 64), (64, 8)):
            rows, cols = split(lib, u, rs, cs, sms)
            check(u, rs, rows)
            check(u, cs, cols)
            whole = sms <= 0 or 2 * u % sms == 0
            if whole:                       # whole waves, or an unknown device: nothing is cut
                assert rows[1] == cols[1] == 1
            elif 2 * u < sms:               # fewer CTAs than SMs: all units of both kernels, alike
                assert rows == cols
            else:                           # the last wave is cols' units alone
                assert rows[1] == 1
                if cols[1] > 1:
                    assert cols[2] == min(u, 2 * u % sms)


def test_pieces_end_sooner(lib):
    """Where units are cut, the last wave takes fewer steps than whole units would, each piece's start counted as ten."""
    for sms in (148, 152):
        for u in range(1, 4 * sms):
            for steps in (16, 25, 64):
                rows, cols = split(lib, u, steps, steps, sms)
                tail, p = 2 * u % sms, cols[1]
                if p > 1:
                    assert -(-tail * p // sms) * (-(-steps // p) + 10) < steps + 10


def test_widths_and_steps(lib):
    for W in range(1, 65):
        w, per = lib.width(W), {16: 4, 32: 2, 48: 1, 64: 1}
        assert W <= w and w in per and w - W < 16
        for H in (1, 2, 3, 4, 5, 31, 64):
            assert lib.rows_steps(H, W) == -(-H // per[w])
