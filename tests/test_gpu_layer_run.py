"""The decoder-layer operators together: one layer of a speculative step in 8
bits, against a 64-bit pass through the same roundings; and how calls share
workspaces, streams and graphs."""
import threading

import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R
import tree_ref as T

pytestmark = pytest.mark.gpu


class Layer:
    """Random 8-bit weights of one decoder layer: attention and a gated
    feed-forward block, norms before and behind each."""

    def __init__(self, c=256, q_heads=4, kv_heads=2, dim=64, f=400, seed=0):
        self.c, self.hq, self.h, self.d, self.f = c, q_heads, kv_heads, dim, f
        g = torch.Generator().manual_seed(seed)

        def weights(m, k):
            return (torch.randint(-127, 128, (m, k), generator=g, dtype=torch.int8).cuda(),
                    (0.015 / k ** 0.5 * torch.exp(0.3 * torch.randn(m, generator=g))).cuda())

        def vector():
            return (1.0 + 0.2 * torch.randn(c, generator=g)).cuda()
        self.qkv, self.back = weights((q_heads + 2 * kv_heads) * dim, c), weights(c, q_heads * dim)
        self.both, self.down = weights(2 * f, c), weights(c, f)
        self.norms = [vector() for _ in range(4)]
        self.freq = torch.from_numpy((1e4 ** (-np.arange(dim // 2) / (dim // 2))).astype(np.float32)).cuda()

    def __call__(self, r, k_cache, v_cache, table, ctx, masks, workspace="auto", stream=None):
        """(residual, next block's input, keys, values) of n nodes per sequence."""
        B, n = masks.shape
        N, kw = B * n, dict(stream=stream)
        bf, i8 = torch.bfloat16, torch.int8

        def new(*shape, dtype=bf):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        x, xs = new(N, self.c, dtype=i8), new(N, dtype=torch.float32)
        vq.residual_norm(r, weight=self.norms[0], out=x, scales_out=xs, **kw)
        rows = vq.gemm_w8a8(*self.qkv, x, xs, new(N, self.qkv[0].shape[0]), workspace=workspace, **kw).view(B, n, -1)
        q, k, v = (t.unflatten(-1, (-1, self.d)) for t in
                   torch.split(rows, [self.hq * self.d, self.h * self.d, self.h * self.d], dim=-1))
        vq.rotate(q, k, self.freq, ctx, tree_mask=masks, q_out=q, k_out=k, **kw)
        seen = vq.tree_attention(q, k, v, k_cache, v_cache, table, ctx, tree_mask=masks, **kw).view(N, -1)
        sq, ss = vq.quant_rows_int8(seen, new(*seen.shape, dtype=i8), new(N, dtype=torch.float32), **kw)
        y = vq.gemm_w8a8(*self.back, sq, ss, new(N, self.c), workspace=workspace, **kw)
        r2 = torch.empty_like(r)
        vq.residual_norm(r, y, self.norms[1], post_weight=self.norms[2], residual_out=r2, out=x, scales_out=xs, **kw)
        f = self.f
        h = vq.gated_w8a8(self.both[0][:f], self.both[1][:f], self.both[0][f:], self.both[1][f:], x, xs, new(N, f),
                          workspace=workspace, **kw)
        hq, hs = vq.quant_rows_int8(h, new(N, f, dtype=i8), new(N, dtype=torch.float32), **kw)
        y = vq.gemm_w8a8(*self.down, hq, hs, new(N, self.c), workspace=workspace, **kw)
        out, r3 = new(N, self.c), torch.empty_like(r)
        vq.residual_norm(r2, y, self.norms[3], residual_out=r3, out=out, alpha=0.5, **kw)
        return r3, out, k, v


def _inputs(layer, B=3, n=7, seed=1):
    g = torch.Generator().manual_seed(seed)
    masks = np.zeros((B, n), np.uint64)
    rs = np.random.RandomState(seed)
    for b in range(B):
        for i in range(n):
            masks[b, i] = (np.uint64(0) if i == 0 else masks[b, rs.randint(i)]) | (np.uint64(1) << np.uint64(i))
    ctx = np.array([0, 33, 70][:B], np.int32)
    P, page = 3 * B, 32
    kc = torch.randn(P, layer.h, page, layer.d, generator=g).to(torch.bfloat16).cuda()
    vc = torch.randn(P, layer.h, page // 32, layer.d, 32, generator=g).to(torch.bfloat16).cuda()
    table = torch.randperm(P, generator=g).to(torch.int32).view(B, 3).cuda()
    r = torch.randn(B * n, layer.c, generator=g).cuda()
    return r, kc, vc, table, torch.from_numpy(ctx).cuda(), torch.from_numpy(masks.view(np.int64)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _bf(a):
    return _np(torch.from_numpy(np.asarray(a, np.float64)).to(torch.bfloat16))


def test_layer_against_64_bits():
    """Every operator's result is rounded as the layer rounds it, so the two
    differ by single roundings that now and then flip: bounded in the mean by a
    few bf16 half steps and 8-bit steps (2^-9 and 1/127 of a row's largest)."""
    L = Layer()
    r, kc, vc, table, ctx, masks = _inputs(L)
    r3, out, _, _ = L(r, kc, vc, table, ctx, masks)
    B, n = masks.shape
    m64 = masks.cpu().numpy().view(np.uint64)
    eps = float(np.float32(1e-6))
    w = [_np(v) for v in L.norms]

    def product(x, xs, pair):
        return R.product(x, xs, pair[0].cpu().numpy(), pair[1].cpu().numpy())[0]
    _, _, h, _ = R.norm(_np(r), None, w[0], None, None, 1.0, eps)
    rows = _bf(product(*R.quant(h), L.qkv)).reshape(B, n, -1)
    q, k, v = (t.reshape(B, n, -1, L.d) for t in np.split(rows, [L.hq * L.d, (L.hq + L.h) * L.d], axis=-1))
    pos = R.positions(ctx.cpu().numpy(), m64, n)
    q, k = (_bf(R.rotate(t, pos, L.freq.cpu().numpy(), False, 1.0)[0]) for t in (q, k))
    seen, _ = T.attention(q, k, v, _np(kc), _np(vc), table.cpu().numpy(), ctx.tolist(), m64, None, L.d ** -0.5, "bf16")
    y = _bf(product(*R.quant(_bf(seen).reshape(B * n, -1)), L.back))
    x, _, h, _ = R.norm(_np(r), y, w[1], w[2], None, 1.0, eps)
    xq = R.quant(h)
    g = L.both[0].cpu().numpy(), L.both[1].cpu().numpy()
    hh = _bf(R.gated(*xq, g[0][:L.f], g[1][:L.f], g[0][L.f:], g[1][L.f:], "silu")[0])
    y = _bf(product(*R.quant(hh), L.down))
    x, _, h, _ = R.norm(x.astype(np.float32).astype(np.float64), y, w[3], None, None, 0.5, eps)
    for got, want in ((r3, x), (out, h)):
        rel = np.linalg.norm(_np(got) - want) / np.linalg.norm(want)
        # in turn: 8 roundings to bf16 (2^-9 each in the mean) and 4 to 8 bits whose
        # flipped codes weigh less, added up
        assert rel <= 8 * 2.0 ** -9 + 4.0 / 127 / 4, rel


def test_layer_streams_graphs_and_workspaces():
    """The same bits on another stream, without workspaces, with one workspace
    shared by all products and with the verify GEMMs, and replayed from a graph
    between eager calls; captured without any call before, too."""
    L = Layer(seed=2)
    args = _inputs(L, seed=5)
    want = [t.clone() for t in L(*args)[:2]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = L(*args)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = L(*args, workspace=None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    shared = vq.Workspace(vq.w8a8_workspace_bytes(1 << 20) + vq.workspace_bytes("q4_0", 4096, 5120))
    codes = torch.randint(0, 256, (4096, 2560), dtype=torch.uint8, device="cuda")
    scales, x = torch.rand(4096, 160, device="cuda").half(), torch.randn(4, 5120, device="cuda").bfloat16()
    plain = vq.gemm_q4_0(codes, scales, x, torch.empty(4, 4096, device="cuda"))
    for _ in range(3):
        got = L(*args, workspace=shared)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        again = vq.gemm_q4_0(codes, scales, x, torch.empty(4, 4096, device="cuda"), workspace=shared)
        assert torch.equal(again, plain)
    for warm in (False, True):
        t = torch.cuda.Stream()
        t.wait_stream(torch.cuda.current_stream())
        if warm:
            with torch.cuda.stream(t):
                L(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=t):
            held = L(*args)
        for _ in range(3):
            held[0].zero_(), held[1].zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])
            with torch.cuda.stream(t):
                got = L(*args)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_host_threads():
    """Threads on one stream and on streams of their own."""
    n, m, k = 100, 3000, 4112
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-127, 128, (m, k), generator=g, dtype=torch.int8).cuda()
    xs, ws = torch.rand(n, generator=g).cuda(), torch.rand(m, generator=g).cuda()
    want = vq.gemm_w8a8(w, ws, x, xs, torch.empty(n, m, device="cuda"), workspace=None)
    torch.cuda.synchronize()
    wrong = []

    def work(stream, rows):
        with torch.cuda.stream(stream):
            for _ in range(40):
                out = vq.gemm_w8a8(w, ws, x[:rows], xs[:rows], torch.empty(rows, m, device="cuda"))
                if not torch.equal(out, want[:rows]):
                    wrong.append(rows)
    same = torch.cuda.Stream()
    ts = [threading.Thread(target=work, args=(same if i < 3 else torch.cuda.Stream(), r))
          for i, r in enumerate((100, 17, 64, 100, 33))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong
