"""Which scratch buffer a call of ``attention``, ``fused`` or ``fused_lse`` gets, with a fake of the CUDA calls."""
from __future__ import annotations

import contextlib

import pytest
import torch

from relative_position_bias_gb300 import api


class Buffer:
    """Stands in for a tensor: a place of its own, and the stream it was allocated on."""
    def __init__(self, n, at, stream):
        self.n, self.at, self.stream = n, at, stream

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


@pytest.fixture
def cuda(monkeypatch):
    """Streams 7 (current) and 8; ``state`` says how much scratch a call needs and which streams are captured."""
    state = dict(need=1000, captured=set(), current=7, made=[])

    def empty(n, **_):
        state["made"].append(Buffer(n, 4096 * (1 + len(state["made"])), state["current"]))
        return state["made"][-1]

    @contextlib.contextmanager
    def stream(s):
        before, state["current"] = state["current"], s.cuda_stream
        yield
        state["current"] = before

    monkeypatch.setattr(api, "_workspaces", {})
    monkeypatch.setattr(api, "workspace_size", lambda *a: state["need"])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(state["current"]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["current"] in state["captured"])
    return state


def get(stream, workspace=None):
    return api._workspace(torch.device("cuda", 0), 12, 64, 64, 64, workspace, stream)


def test_eager_calls_of_a_stream_share_a_buffer(cuda):
    a, b, other = get(7), get(7), get(8)
    assert a[-2:] == b[-2:] == (4096, 1000) and other[-2] != a[-2]
    cuda["need"] = 2000
    assert get(7)[-2:] == (cuda["made"][-1].at, 2000)
    cuda["need"] = 500
    assert get(7)[-2:] == (cuda["made"][-1].at, 2000)     # a larger one serves
    assert [m.stream for m in cuda["made"]] == [7, 8, 7]   # each of the stream that uses it


def test_captured_calls_have_buffers_of_their_own(cuda):
    """Two graphs captured on one stream may be replayed at the same time, and long after the eager calls of that
    stream have taken a larger buffer."""
    eager = get(7)
    cuda["captured"] = {7}
    first, second = get(7), get(7)
    assert len({eager[-2], first[-2], second[-2]}) == 3 and first[-1] == second[-1] == 1000
    assert isinstance(first[0], Buffer)                   # the caller holds it until the launch
    cuda["captured"] = set()
    assert get(7)[-2] == eager[-2]
    cuda["captured"] = {8}                                # captured, but not the current stream
    side = get(8)
    assert side[-2] == cuda["made"][-1].at and cuda["made"][-1].stream == 8
    assert get(7)[-2] == eager[-2]


def test_no_scratch(cuda):
    cuda["captured"] = {7}
    assert get(7, workspace=False)[-2:] == (None, 0)
    cuda["need"] = 0
    assert get(7)[-2:] == (None, 0) and not cuda["made"]
