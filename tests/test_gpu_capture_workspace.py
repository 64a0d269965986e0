"""Default workspaces that are made while a graph is captured: zeroed once, now,
and not by the graph's replays; the capture goes on; calls before, between and
after the replays are right."""
import pytest
import torch

import block_quantized_gemm_amd as vq
import plan_host as H

pytestmark = pytest.mark.gpu


def _codes(n, m, k, seed):
    g = torch.Generator().manual_seed(seed)
    x, w = (torch.randint(-127, 128, (r, k), generator=g, dtype=torch.int8).cuda() for r in (n, m))
    return w, torch.rand(m, generator=g).cuda() / k, x, torch.rand(n, generator=g).cuda()


def _plain(n, m, k):
    w, ws, x, xs = _codes(n, m, k, n)
    assert H.plan(n, m, k, cus=torch.cuda.get_device_properties(0).multi_processor_count).cuts > 1
    out = torch.empty(n, m, device="cuda")
    return lambda **kw: vq.gemm_w8a8(w, ws, x, xs, out, **kw), out


def _gated(n, f, k):
    w, ws, x, xs = _codes(n, 2 * f, k, n)
    assert H.plan(n, f, k, True, cus=torch.cuda.get_device_properties(0).multi_processor_count).cuts > 1
    out = torch.empty(n, f, device="cuda")
    return lambda **kw: vq.gated_w8a8(w[:f], ws[:f], w[f:], ws[f:], x, xs, out, **kw), out


def _q4_0(n, m, k):
    g = torch.Generator().manual_seed(n)
    codes = torch.randint(0, 256, (m, k // 2), generator=g, dtype=torch.uint8).cuda()
    scales, x = torch.rand(m, k // 32, generator=g).half().cuda(), torch.randn(n, k, generator=g).bfloat16().cuda()
    assert vq.default_launch_shape("q4_0", m, k)[2] == 1  # the walk form, with its counters
    out = torch.empty(n, m, device="cuda")
    return lambda **kw: vq.gemm_q4_0(codes, scales, x, out, **kw), out


CALLS = [(_plain, 98, 2633, 6240), (_plain, 227, 2101, 4176), (_gated, 99, 1307, 6736), (_gated, 67, 4561, 5776),
         (_q4_0, 4, 4096, 5120)]


def _fresh_stream():
    """A stream that no earlier call has had (torch hands them out in turn)."""
    for _ in range(64):
        s = torch.cuda.Stream()
        if not any(key[-1] == s.cuda_stream for key in vq._auto_ws):
            return s
    vq._auto_ws.clear()
    return s


def _of(stream):
    return [ws for key, ws in vq._auto_ws.items() if key[-1] == stream.cuda_stream]


@pytest.mark.parametrize("make,n,m,k", CALLS)
def test_first_call_is_captured(make, n, m, k):
    call, out = make(n, m, k)
    want = call().clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    ws, = _of(s)
    assert not ws.tensor.any(), "zeroed when it was made"
    with torch.cuda.stream(s):  # before any replay
        out.fill_(-1)
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    used, counters = ws.tensor.any().item(), ws.tensor[:H.lib().counter_bytes()]
    assert used and not counters.any()
    mark = make is not _q4_0  # (their workspaces hold more than these forms use)
    for _ in range(4):
        out.fill_(-1)
        if mark:
            ws.tensor[-1] = 77
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not counters.any()
        assert not mark or ws.tensor[-1] == 77, "a replay clears the workspace"
        out.fill_(-1)
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("make,n,m,k", CALLS)
def test_captured_stream_that_is_not_current(make, n, m, k):
    """The stream is given to the call; another is current."""
    call, out = make(n, m, k)
    want = call().clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin()
    try:
        call(stream=s)
    finally:
        with torch.cuda.stream(s):
            graph.capture_end()
    for _ in range(3):
        out.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_graphs_of_two_streams_overlap():
    """Captured on streams of their own, without a call before: each has its workspace."""
    made = [make(n, m, k) for make, n, m, k in CALLS[:2]]
    want = [call().clone() for call, _ in made]
    streams, graphs = [], []
    for call, out in made:
        s = _fresh_stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(20):
                call()
        streams.append(s)
        graphs.append(g)
    assert _of(streams[0])[0].ptr() != _of(streams[1])[0].ptr()
    for _ in range(5):
        for _, out in made:
            out.fill_(-1)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for (_, out), w in zip(made, want))
