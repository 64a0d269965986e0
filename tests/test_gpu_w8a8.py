"""The 8-bit products against 64-bit definitions: sizes around every tile
border, extreme codes and sums, every output type, the same bits for any
number of rows."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(n, m, k, seed, lo=-128, hi=128):
    g = np.random.Generator(np.random.PCG64(seed))
    x, w = g.integers(lo, hi, (n, k)).astype(np.int8), g.integers(lo, hi, (m, k)).astype(np.int8)
    # sums are about 5,500 sqrt(k): scales that make outputs of about 1, some channels and rows far from it
    xs = (0.01 * np.exp(g.standard_normal(n))).astype(np.float32)
    ws = (0.02 / np.sqrt(k) * np.exp(g.standard_normal(m))).astype(np.float32)
    return x, xs, w, ws, g.standard_normal(m).astype(np.float32)


def _dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def _close(got, y, err, out):
    off = np.abs(got.double().cpu().numpy() - y)
    worst = (off / R.rounded(y, err, out)).max()
    assert worst <= 1.0, worst


SIZES = [(1, 1, 16), (1, 5, 16), (2, 16, 32), (3, 17, 48), (5, 127, 112), (15, 128, 128), (16, 129, 144), (17, 130, 240),
         (16, 2001, 256), (33, 255, 272), (48, 257, 1040), (63, 64, 512), (64, 512, 640), (65, 300, 384), (127, 256, 896),
         (129, 511, 1296), (200, 258, 2064), (256, 1028, 528), (257, 516, 4112), (300, 77, 1024), (513, 1023, 320)]


@pytest.mark.parametrize("n,m,k", SIZES)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_product(n, m, k, out):
    x, xs, w, ws, bias = _case(n, m, k, 7 * n + m + k)
    dx, dxs, dw, dws, db = _dev(x, xs, w, ws, bias)
    got = vq.gemm_w8a8(dw, dws, dx, dxs, torch.full((n, m), float("nan"), dtype=DT[out], device="cuda"))
    _close(got, *R.product(x, xs, w, ws), out)
    got = vq.gemm_w8a8(dw, dws, dx, dxs, torch.full((n, m), float("nan"), dtype=DT[out], device="cuda"), bias=db)
    _close(got, *R.product(x, xs, w, ws, bias), out)


@pytest.mark.parametrize("n,f,k", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated(n, f, k, act):
    x, xs, w, ws, _ = _case(n, 2 * f, k, 3 * n + f + k)
    out = ["bf16", "f16", "f32"][(n + f) % 3]
    dx, dxs, dw, dws = _dev(x, xs, w, ws)
    got = vq.gated_w8a8(dw[:f], dws[:f], dw[f:], dws[f:], dx, dxs,
                        torch.full((n, f), float("nan"), dtype=DT[out], device="cuda"), activation=act)
    _close(got, *R.gated(x, xs, w[:f], ws[:f], w[f:], ws[f:], act), out)


@pytest.mark.parametrize("n", [1, 7, 16, 40, 70, 300])
@pytest.mark.parametrize("code", [(-128, -128), (127, -128), (127, 127)])
def test_largest_sums(n, code):
    """Every term the same extreme product, over the longest row: 131056 * 2^14
    is the largest sum that 32 bits hold."""
    m, k = 40, vq_max_k()
    x, w = np.full((n, k), code[0], np.int8), np.full((m, k), code[1], np.int8)
    dx, dw = _dev(x, w)
    one = torch.ones(max(n, m), device="cuda")
    got = vq.gemm_w8a8(dw, one[:m], dx, one[:n], torch.zeros(n, m, device="cuda"))
    want = np.float32(k * code[0] * code[1])
    assert (got.cpu().numpy() == want).all()


def vq_max_k():
    return 131056


@pytest.mark.parametrize("m,k", [(300, 1040), (1000, 5120), (4096, 144)])
def test_rows_do_not_depend_on_their_number(m, k):
    n = 530
    x, xs, w, ws, bias = _case(n, 2 * m, k, 5)
    dx, dxs, dw, dws, db = _dev(x, xs, w, ws, bias)
    whole = vq.gemm_w8a8(dw, dws, dx, dxs, torch.empty(n, 2 * m, device="cuda"), bias=db)
    both = vq.gated_w8a8(dw[:m], dws[:m], dw[m:], dws[m:], dx, dxs, torch.empty(n, m, device="cuda"))
    for rows in (1, 2, 16, 17, 32, 64, 65, 100, 128, 129, 255, 256, 400):
        for ws_arg in ("auto", None):
            part = vq.gemm_w8a8(dw, dws, dx[:rows], dxs[:rows], torch.empty(rows, 2 * m, device="cuda"), bias=db,
                                workspace=ws_arg)
            assert torch.equal(part, whole[:rows]), (rows, ws_arg)
            part = vq.gated_w8a8(dw[:m], dws[:m], dw[m:], dws[m:], dx[:rows], dxs[:rows],
                                 torch.empty(rows, m, device="cuda"), workspace=ws_arg)
            assert torch.equal(part, both[:rows]), (rows, ws_arg)


@pytest.mark.parametrize("n,m", [(1, 33), (16, 128), (50, 130), (130, 257), (300, 640)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_nothing_else_is_written(n, m, out):
    k = 272
    x, xs, w, ws, _ = _case(n, 2 * m, k, 11)
    dx, dxs, dw, dws = _dev(x, xs, w, ws)
    for gated in (False, True):
        around = torch.full((n * m + 512,), 3.0, dtype=DT[out], device="cuda")
        mid = around[256:256 + n * m].view(n, m)
        if gated:
            vq.gated_w8a8(dw[:m], dws[:m], dw[m:], dws[m:], dx, dxs, mid)
        else:
            vq.gemm_w8a8(dw[:m], dws[:m], dx, dxs, mid)
        assert (around[:256] == 3).all() and (around[256 + n * m:] == 3).all()


def test_scales_pass_through():
    """A NaN or infinite scale shows in its row or channel alone; zeros too."""
    n, m, k = 20, 70, 64
    x, xs, w, ws, _ = _case(n, m, k, 13)
    x[:, 0], w[:, 0] = 127, 127
    xs[3], ws[5], xs[4] = np.nan, np.inf, 0.0
    dx, dxs, dw, dws = _dev(x, xs, w, ws)
    got = vq.gemm_w8a8(dw, dws, dx, dxs, torch.empty(n, m, device="cuda")).cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = ((x.astype(np.int64) @ w.astype(np.int64).T).astype(np.float32) * xs[:, None]) * ws
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("n", [1, 16, 61, 200])
def test_captured_and_replayed(n):
    """A graph of both products, replayed with eager calls of other sizes in between."""
    m, k = 1100, 2064
    x, xs, w, ws, _ = _case(n, 2 * m, k, 17)
    dx, dxs, dw, dws = _dev(x, xs, w, ws)
    s = torch.cuda.Stream()
    a, b = torch.empty(n, 2 * m, device="cuda"), torch.empty(n, m, device="cuda")

    def both():
        vq.gemm_w8a8(dw, dws, dx, dxs, a)
        vq.gated_w8a8(dw[:m], dws[:m], dw[m:], dws[m:], dx, dxs, b)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.synchronize()
    want = a.clone(), b.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for i in range(4):
        a.zero_(), b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        with torch.cuda.stream(s):
            vq.gemm_w8a8(dw[:700], dws[:700], dx[:1], dxs[:1], torch.empty(1, 700, device="cuda"))
        torch.cuda.synchronize()


def test_binding_checks():
    x, xs, w, ws, _ = _case(4, 32, 64, 1)
    dx, dxs, dw, dws = _dev(x, xs, w, ws)
    out = torch.empty(4, 32, device="cuda")
    for bad in (dict(w=dw[:, ::2]), dict(x=dx.t().contiguous().t()), dict(ws=dws.double()), dict(xs=dxs[:3]),
                dict(x=dx.int()), dict(out=out.t().contiguous().t()), dict(ws=dws.cpu())):
        a = dict(w=dw, ws=dws, x=dx, xs=dxs, out=out) | bad
        with pytest.raises((ValueError, TypeError)):
            vq.gemm_w8a8(a["w"], a["ws"], a["x"], a["xs"], a["out"])
    with pytest.raises(ValueError, match="share"):
        vq.gemm_w8a8(dw, dws, dx, dxs, dw.view(-1)[:512].view(torch.float32).view(4, 32))
    with pytest.raises(vq.VqError):
        vq.gemm_w8a8(dw[:, :24].contiguous(), dws, dx[:, :24].contiguous(), dxs, out)


@pytest.mark.parametrize("n,m,k", [(300007, 21, 32), (3, 400009, 64), (70001, 70000, 16)])
def test_many_rows_and_features(n, m, k):
    """Long sides, and outputs whose offsets pass 32 bits: sampled rows and columns."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones(max(n, m), device="cuda")
    out = vq.gemm_w8a8(w, one[:m], x, one[:n], torch.empty(n, m, dtype=torch.bfloat16, device="cuda"))
    rows = torch.tensor(sorted({0, 1, n // 2, n - 2 if n > 1 else 0, n - 1}), device="cuda")
    cols = torch.tensor(sorted({0, m // 3, m - 1, m - 2}), device="cuda")
    want = x[rows].double() @ w.double().t().contiguous()  # whole numbers below 2^24: one rounding to bf16
    assert torch.equal(out[rows], want.to(torch.bfloat16))
    want = x.double() @ w[cols].double().t().contiguous()
    assert torch.equal(out[:, cols], want.to(torch.bfloat16))
