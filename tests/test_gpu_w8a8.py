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


# (rows, features, k): on 256 compute units these reach every form of the
# kernel, with tiles whole, in several rounds, and cut in two, three and more
PLAIN = [(1, 33, 4144), (1, 1485, 5696), (17, 16889, 1568), (18, 16883, 4112), (17, 17435, 144), (17, 22395, 3728),
         (17, 17401, 5072), (18, 6885, 144), (18, 17067, 224), (1178, 65, 8720), (935, 33, 7584), (33, 11535, 144),
         (34, 5279, 6928), (98, 2633, 6240), (66, 8215, 144), (131, 16677, 144), (227, 2101, 4176), (325, 5405, 144),
         (716, 5381, 144), (199, 3949, 7488), (99, 4359, 4624), (66, 16807, 144), (257, 17083, 144), (66, 9273, 6352),
         (269, 15471, 5680), (68, 8359, 5680), (264, 11209, 8224), (134, 21853, 144), (653, 22055, 144), (199, 8507, 5312),
         (258, 22397, 144), (401, 8333, 7056), (1300, 6001, 1040)]
GATED = [(1, 33, 4144), (1, 16453, 400), (1, 737, 5728), (1, 17125, 5936), (1, 16469, 4192), (1, 8195, 144),
         (17, 18887, 1680), (18, 17485, 1648), (19, 3387, 144), (17, 8903, 224), (1284, 35, 8000), (615, 33, 7200),
         (33, 5449, 144), (36, 21099, 2272), (33, 3273, 5584), (99, 1307, 6736), (66, 4223, 144), (35, 16503, 144),
         (33, 21095, 1936), (163, 1375, 4144), (33, 16975, 1888), (1219, 773, 144), (1273, 1609, 208), (193, 1935, 8048),
         (66, 19033, 1968), (101, 2085, 4752), (69, 16559, 1952), (66, 8215, 144), (66, 16807, 144), (67, 4561, 5776),
         (65, 21137, 3120), (194, 2155, 3728), (67, 19055, 3040), (133, 11069, 144), (258, 22397, 144), (577, 13061, 1936),
         (197, 4155, 5424), (386, 17053, 2016), (131, 16677, 144), (517, 17321, 144), (386, 4313, 6816)]


def _device_case(n, m, k):
    g = torch.Generator(device="cuda").manual_seed(n * 31 + m + k)
    x, w = (torch.randint(-128, 128, (r, k), generator=g, device="cuda", dtype=torch.int8) for r in (n, m))
    xs = 0.01 * torch.exp(torch.randn(n, generator=g, device="cuda"))
    return x, xs, w, 0.02 / k ** 0.5 * torch.exp(torch.randn(m, generator=g, device="cuda"))


@pytest.mark.parametrize("n,m,k", PLAIN)
def test_every_form(n, m, k):
    """The definition's own operations, bit for bit: the exact sum, to fp32,
    times the row's scale, times the channel's; twice, so that the counters of
    cut tiles are seen to be back at zero, and without a workspace."""
    x, xs, w, ws = _device_case(n, m, k)
    dots = x.double() @ w.double().t().contiguous()  # exact in 64 bits
    want = dots.float() * xs[:, None] * ws
    for out, workspace in (("f32", "auto"), ("bf16", "auto"), ("f16", None)):
        got = vq.gemm_w8a8(w, ws, x, xs, torch.full((n, m), float("nan"), dtype=DT[out], device="cuda"),
                           workspace=workspace)
        assert torch.equal(got, want.to(DT[out])), out


@pytest.mark.parametrize("n,f,k", GATED)
def test_every_gated_form(n, f, k):
    """The rows as the form for few rows gives them, which the tests above hold
    to the definition, bit for bit; and the definition in 64 bits."""
    x, xs, w, ws = _device_case(n, 2 * f, k)
    act = ["silu", "gelu", "gelu_tanh"][(n + f) % 3]

    def call(rows, workspace="auto"):
        return vq.gated_w8a8(w[:f], ws[:f], w[f:], ws[f:], x[rows], xs[rows],
                             torch.full((len(xs[rows]), f), float("nan"), device="cuda"), activation=act,
                             workspace=workspace)
    whole = call(slice(None))
    assert torch.equal(whole, call(slice(None))) and torch.equal(whole, call(slice(None), None))
    for at in range(0, n, max(16, n // 6 // 16 * 16)):
        assert torch.equal(whole[at:at + 16], call(slice(at, at + 16))), at
    # the sum before the scales: it is an integer, 0 where the terms cancel
    both = (x.double() @ w.double().t().contiguous()) * xs.double()[:, None] * ws.double()
    g, u = both[:, :f], both[:, f:]
    if act == "silu":
        want = g * torch.sigmoid(g) * u
    elif act == "gelu":
        want = 0.5 * g * torch.special.erfc(g * -0.5 ** 0.5) * u
    else:
        z = (2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)
        want = g * torch.sigmoid(2 * z) * u
    # sums of 1.1 |g| 3 U, 3 U of u and the activation's own (R.activate), the largest of the three kinds
    bound = R.U * (3.4 * g.abs() * u.abs() + (60 + 24 * g.abs() ** 3 + 4 * g * g) * want.abs()) + 1e-37 * (1 + u.abs())
    assert bool(((whole.double() - want).abs() <= bound).all())
