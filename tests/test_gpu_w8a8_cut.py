"""The 8-bit products where tiles are cut between workgroups: what streams,
graphs, host threads and other operators share a workspace with; and every form
with guards around its outputs, with a bias, in every type."""
import threading

import pytest
import torch

import block_quantized_gemm_amd as vq
import plan_host as H
import test_gpu_w8a8 as G
from single_rounding import fma

pytestmark = pytest.mark.gpu
DT = G.DT


def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


class Product:
    """A product whose plan is cut (asserted), its result without a workspace,
    and calls of its first rows."""

    def __init__(self, n, m, k, gated):
        p = H.plan(n, m, k, gated, cus=_cus())
        assert p.cuts > 1, (n, m, k, p)
        self.n, self.m, self.gated = n, m, gated
        x, xs, w, ws = G._device_case(n, (2 if gated else 1) * m, k)
        self.x, self.xs, self.w, self.ws = x, xs, w, ws
        self.want = self(workspace=None)

    def __call__(self, out=None, **kw):
        out = torch.full((self.n, self.m), float("nan"), device="cuda") if out is None else out
        if self.gated:
            return vq.gated_w8a8(self.w[:self.m], self.ws[:self.m], self.w[self.m:], self.ws[self.m:], self.x, self.xs,
                                 out, **kw)
        return vq.gemm_w8a8(self.w, self.ws, self.x, self.xs, out, **kw)


CUT = [(98, 2633, 6240, False), (227, 2101, 4176, False), (99, 1307, 6736, True), (67, 4561, 5776, True),
       (1178, 65, 8720, False), (193, 1935, 8048, True)]
IDS = ["%s-%d-%d-%d" % ("gated" if c[3] else "plain", *c[:3]) for c in CUT]


def _workspace():
    return vq.Workspace(vq.w8a8_workspace_bytes(1 << 20))


def _counters(ws):
    return ws.tensor[:H.lib().counter_bytes()]


def _check_used(ws):
    """Sums have gone through the buffer, and its counters are back at zero."""
    torch.cuda.synchronize()
    assert ws.tensor[H.lib().counter_bytes():].any() and not _counters(ws).any()


@pytest.mark.parametrize("case", CUT, ids=IDS)
def test_one_workspace_in_turn(case):
    """Another stream; the same workspace for products of other sizes and for
    the verify GEMMs, in any order."""
    p, other = Product(*case), Product(*CUT[(CUT.index(case) + 2) % len(CUT)])
    ws = _workspace()
    codes = torch.randint(0, 256, (4096, 2560), dtype=torch.uint8, device="cuda")
    scales, x = torch.rand(4096, 160, device="cuda").half(), torch.randn(4, 5120, device="cuda").bfloat16()
    assert vq.default_launch_shape("q4_0", 4096, 5120)[2] == 1
    verify = vq.gemm_q4_0(codes, scales, x, torch.empty(4, 4096, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        with torch.cuda.stream(s if i % 2 else torch.cuda.current_stream()):
            assert torch.equal(p(workspace=ws), p.want), i
            _check_used(ws)
            ws.tensor[H.lib().counter_bytes():].fill_(0xA5)  # (pieces may hold anything)
            assert torch.equal(other(workspace=ws), other.want), i
            _check_used(ws)
            again = vq.gemm_q4_0(codes, scales, x, torch.empty(4, 4096, device="cuda"), workspace=ws)
            assert torch.equal(again, verify), i
            _check_used(ws)
            torch.cuda.synchronize()


@pytest.mark.parametrize("case", CUT, ids=IDS)
@pytest.mark.parametrize("kind", ["auto", "own"])
def test_captured_and_replayed(case, kind):
    """Replays with eager calls of this product and of another one between
    them, all through one workspace."""
    p, other = Product(*case), Product(*CUT[(CUT.index(case) + 1) % len(CUT)])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = _workspace() if kind == "own" else "auto"
    a, b = torch.empty(p.n, p.m, device="cuda"), torch.empty(other.n, other.m, device="cuda")
    with torch.cuda.stream(s):
        p(a, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p(a, workspace=ws)
        other(b, workspace=ws)
        p(a, workspace=ws)
    if kind == "auto":
        key, = [k for k in vq._auto_ws if k[0] == "vq_w8a8_workspace_bytes" and k[-1] == s.cuda_stream]
        ws = vq._auto_ws[key]
    for i in range(4):
        a.fill_(-1), b.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        _check_used(ws)
        assert torch.equal(a, p.want) and torch.equal(b, other.want), i
        with torch.cuda.stream(s):
            assert torch.equal(other(workspace=ws), other.want) and torch.equal(p(workspace=ws), p.want), i
        _check_used(ws)


def test_host_threads():
    """Three threads on one stream, two on streams of their own, each with a
    product of its own, default workspaces."""
    made = [Product(*c) for c in CUT[:5]]
    torch.cuda.synchronize()
    same, wrong = torch.cuda.Stream(), []
    streams = [same, same, same, torch.cuda.Stream(), torch.cuda.Stream()]

    def work(p, stream):
        with torch.cuda.stream(stream):
            for _ in range(40):
                if not torch.equal(p(), p.want):
                    wrong.append((p.n, p.m))
    threads = [threading.Thread(target=work, args=a) for a in zip(made, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for key, ws in vq._auto_ws.items():
        if key[0] == "vq_w8a8_workspace_bytes" and key[-1] in {s.cuda_stream for s in streams}:
            _check_used(ws)


def _guarded(n, m, out):
    """(buffer, the [n][m] array within it): 256 elements on each side."""
    around = torch.full((n * m + 512,), 3.0, dtype=DT[out], device="cuda")
    mid = around[256:256 + n * m].view(n, m)
    mid.fill_(float("nan"))
    return around, mid


def _untouched(around):
    return bool((around[:256] == 3).all() and (around[-256:] == 3).all())


@pytest.mark.parametrize("n,m,k", G.PLAIN)
def test_every_form_between_guards(n, m, k):
    """Bit for bit with a bias, in every type, with a workspace and without;
    nothing beside the outputs is written."""
    x, xs, w, ws = G._device_case(n, m, k)
    bias = torch.randn(m, generator=torch.Generator(device="cuda").manual_seed(m), device="cuda")
    scaled = (x.double() @ w.double().t().contiguous()).float() * xs[:, None]
    for b, want in ((None, scaled * ws), (bias, fma(scaled, ws[None], bias[None]))):
        for out in ("f32", "bf16", "f16"):
            for workspace in ("auto", None):
                around, mid = _guarded(n, m, out)
                vq.gemm_w8a8(w, ws, x, xs, mid, bias=b, workspace=workspace)
                assert torch.equal(mid, want.to(DT[out])) and _untouched(around), (out, workspace, b is None)


@pytest.mark.parametrize("n,f,k", G.GATED)
def test_every_gated_form_between_guards(n, f, k):
    """The same bits with a workspace and without in every type, and nothing
    beside the outputs is written.  (The values are held to the definition in the
    tests of every gated form.)"""
    x, xs, w, ws = G._device_case(n, 2 * f, k)
    for out in ("f32", "bf16", "f16"):
        for act in ("silu", "gelu", "gelu_tanh"):
            got = []
            for workspace in ("auto", None):
                around, mid = _guarded(n, f, out)
                vq.gated_w8a8(w[:f], ws[:f], w[f:], ws[f:], x, xs, mid, activation=act, workspace=workspace)
                assert _untouched(around), (out, act, workspace)
                got.append(mid)
            assert torch.equal(*got) and not torch.isnan(got[0]).any(), (out, act)

