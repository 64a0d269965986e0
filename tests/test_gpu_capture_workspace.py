"""Default workspaces that are first needed while a graph is captured: the
8-bit products get one of the graph's own, the verify GEMMs the stream's, zeroed
outside the graph; the capture goes on; calls before, between and after the
replays are right."""
import ctypes

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


def _graph_workspace(stream):
    return vq._graph_ws[(torch.device("cuda", 0), stream.cuda_stream)][1]


@pytest.mark.parametrize("make,n,m,k", CALLS[:4])
def test_first_product_is_captured(make, n, m, k):
    call, out = make(n, m, k)
    want = call().clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
        call()
        other = torch.full((1 << 22,), 5, dtype=torch.int32, device="cuda")  # the graph's, not over the workspace
    assert not _of(s)  # eager calls have none of it
    buffer = _graph_workspace(s)
    counters = buffer[:H.lib().counter_bytes()]
    for i in range(4):
        out.fill_(-1)
        counters.fill_(0xFF)  # whatever ended in between: the graph clears them
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not counters.any() and buffer.any() and (other == 5).all(), i
        out.fill_(-1)
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and not counters.any(), i
    assert len(_of(s)) == 1 and _of(s)[0].ptr() != buffer.data_ptr()


def test_a_product_that_is_not_cut_needs_none():
    w, ws, x, xs = _codes(1, 5120, 1024, 3)
    assert vq.w8a8_workspace_used(1, 5120, 1024) == 0
    out = torch.empty(1, 5120, device="cuda")
    want = vq.gemm_w8a8(w, ws, x, xs, out).clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    graph, before = torch.cuda.CUDAGraph(), dict(vq._graph_ws)
    with torch.cuda.graph(graph, stream=s):
        vq.gemm_w8a8(w, ws, x, xs, out)
    assert vq._graph_ws == before and not _of(s)
    out.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_graphs_of_one_stream_overlap():
    """Captured one after the other on one stream, as torch does by default,
    without a call before; the second needs more. Replayed at once on two streams,
    also after the second capture has let go of the first one's buffer."""
    made = [make(n, m, k) for make, n, m, k in (CALLS[3], CALLS[0], CALLS[1])]
    want = [call().clone() for call, _ in made]
    s, graphs = _fresh_stream(), []
    for call, out in made:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(20):
                call()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        for _, out in made:
            out.fill_(-1)
        filled = [torch.full((1 << 20,), 0x3C, dtype=torch.uint8, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        for t, g in zip(streams, graphs):
            with torch.cuda.stream(t):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for (_, out), w in zip(made, want))
        assert all(bool((f == 0x3C).all()) for f in filled)


def test_a_larger_call_in_one_capture():
    (small, a), (large, b) = _plain(98, 2633, 6240), _plain(227, 2101, 4176)
    want = small().clone(), large().clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        small(), large(), small()
    for _ in range(4):
        a.fill_(-1), b.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_capture_that_is_not_of_torch():
    """Through the runtime itself: no memory of a graph's own, so no workspace."""
    call, out = _plain(98, 2633, 6240)
    want = call().clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    P, pp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)
    graph, made = P(), P()
    assert vq._hip("hipStreamBeginCapture", P, ctypes.c_int)(s.cuda_stream, 0) == 0
    try:
        call(stream=s)
    finally:
        assert vq._hip("hipStreamEndCapture", P, pp)(s.cuda_stream, ctypes.byref(graph)) == 0
    assert (torch.device("cuda", 0), s.cuda_stream) not in vq._graph_ws and not _of(s)
    assert vq._hip("hipGraphInstantiate", pp, P, P, P, ctypes.c_size_t)(ctypes.byref(made), graph, None, None, 0) == 0
    for _ in range(3):
        out.fill_(-1)
        torch.cuda.synchronize()
        assert vq._hip("hipGraphLaunch", P, P)(made, s.cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert vq._hip("hipGraphExecDestroy", P)(made) == 0 and vq._hip("hipGraphDestroy", P)(graph) == 0


def test_first_verify_gemm_is_captured():
    call, out = _q4_0(4, 4096, 5120)
    want = call().clone()
    s = _fresh_stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    ws, = _of(s)
    assert not ws.tensor.any(), "zeroed when it was made"
    counters = ws.tensor[:H.lib().counter_bytes()]
    with torch.cuda.stream(s):  # before any replay
        out.fill_(-1)
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ws.tensor.any() and not counters.any()
    for _ in range(4):
        for run in (graph.replay, call):
            out.fill_(-1)
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                run()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and not counters.any()


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
