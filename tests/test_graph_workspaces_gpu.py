"""Captured calls of the entries whose units are cut: graphs share no scratch with one another or with eager calls."""
from __future__ import annotations

import pytest
import torch

import relative_position_bias_gb300 as rpb
from relative_position_bias_gb300 import build as rbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()
    rpb.load_library()
    yield
    assert rpb.device_status() == 0, "a kernel hit its bounded-wait budget"


def call(entry, x):
    if entry == "attention":
        return (rpb.attention(x["q"], x["k"], x["v"], x["rh"], x["rw"], 64, 64),)
    if entry == "fused":
        return (rpb.fused(x["q"], x["k"], x["v"], x["th"], x["tw"], 64, 64),)
    return rpb.fused_lse(x["q"], x["k"], x["v"], x["th"], x["tw"], 64, 64)


def make(BH, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = {n: torch.randn(BH, 4096, 64, generator=g, device="cuda").bfloat16() for n in ("q", "k", "v")}
    x |= {n: torch.randn(BH, 4096, 64, generator=g, device="cuda") for n in ("rh", "rw")}
    return x | {n: 0.3 * torch.randn(127, 64, generator=g, device="cuda").bfloat16() for n in ("th", "tw")}


@pytest.mark.parametrize("entry", ["attention", "fused", "fused_lse"])
def test_graphs_of_one_stream_side_by_side(entry):
    """Two graphs captured on one stream after eager calls there, replayed at the same time on two streams while a larger
    eager call runs on a third."""
    xs, large = [make(12, s) for s in (1, 2)], make(44, 3)
    assert rpb.workspace_size(12, 64, 64) > 0 and rpb.workspace_size(44, 64, 64) > 0
    want = [call(entry, x) for x in xs]
    want_large = call(entry, large)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, res = [], []
    with torch.cuda.stream(side):
        call(entry, xs[0])                       # the stream's eager buffer, of the smaller size
    torch.cuda.synchronize()
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            res.append(call(entry, x))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for r in res:
            for t in r:
                t.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(side):
            got = call(entry, large)
        torch.cuda.synchronize()
        for a, b in zip([*res, got], [*want, want_large]):
            assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("entry", ["attention", "fused"])
def test_captured_stream_that_is_not_the_current_one(entry):
    """A call into the caller's output whose stream is captured while another is current: its scratch is the graph's, not
    memory that is handed out again once the call has returned."""
    x = make(12, 4)
    out = torch.empty_like(x["q"])

    def run(**more):
        bias = (x["rh"], x["rw"]) if entry == "attention" else (x["th"], x["tw"])
        return getattr(rpb, entry)(x["q"], x["k"], x["v"], *bias, 64, 64, **more)
    want = run()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with torch.cuda.stream(other):
            run(out=out, stream=side)
    taken = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(32)]   # what freed memory would go to
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(t.isnan().all() for t in taken)
