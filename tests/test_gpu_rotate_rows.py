"""The rotation of queries and keys against a 64-bit definition: layouts, part
of the head, far positions, trees, strided rows, in place."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _fused(B, n, hq, h, d, dt, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    m = torch.randn(B, n, (hq + 2 * h) * d + pad, generator=g).to(DT[dt]).cuda()
    q, k, v, _ = torch.split(m, [hq * d, h * d, h * d, pad], dim=-1)
    return m, q.unflatten(-1, (hq, d)), k.unflatten(-1, (h, d)), v


def _freq(rot, base=1e6, stretch=1.0):
    return (base ** (-2.0 * np.arange(rot // 2) / rot) / stretch).astype(np.float32)


def _check(got, t, pos, freq, interleaved, scale, dt):
    y, err = R.rotate(t.double().cpu().numpy(), pos, freq, interleaved, scale)
    off = np.abs(got.double().cpu().numpy() - y)
    # channels that only pass through are copied
    bound = np.where(err > 0, R.rounded(y, err, dt), np.where(off > 0, 0, 1))
    assert (off <= bound).all()


def _masks(B, n, seed):
    g = np.random.RandomState(seed)
    m = np.zeros((B, n), np.uint64)
    for b in range(B):
        for i in range(n):
            m[b, i] = (np.uint64(0) if i == 0 else m[b, g.randint(i)]) | (np.uint64(1) << np.uint64(i))
    return m


@pytest.mark.parametrize("B,n,hq,h,d,rot", [(1, 1, 1, 1, 64, 64), (2, 3, 8, 2, 128, 128), (3, 64, 6, 6, 128, 64),
                                            (1, 7, 5, 1, 256, 64), (2, 5, 64, 8, 128, 16), (1, 2, 3, 3, 16, 16),
                                            (2, 9, 2, 1, 80, 48), (1, 2, 1, 1, 512, 512)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(B, n, hq, h, d, rot, dt, interleaved):
    m, q, k, _ = _fused(B, n, hq, h, d, dt, B * n + d, pad=8)
    freq = _freq(rot)
    ctx = np.array([0, 40961, 1000000][:B], np.int32)
    f, c = torch.from_numpy(freq).cuda(), torch.from_numpy(ctx).cuda()
    before = m.clone()
    for masks in (None, _masks(B, n, d)):
        tm = None if masks is None else torch.from_numpy(masks.view(np.int64)).cuda()
        pos = R.positions(ctx, masks, n)
        qo, ko = vq.rotate(q, k, f, c, tree_mask=tm, interleaved=interleaved, scale=1.25)
        assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(m, before)
        _check(qo, q, pos, freq, interleaved, float(np.float32(1.25)), dt)
        _check(ko, k, pos, freq, interleaved, float(np.float32(1.25)), dt)
        alone, none = vq.rotate(q, None, f, c, tree_mask=tm, interleaved=interleaved, scale=1.25)
        assert none is None and torch.equal(alone, qo)
        # in place, within the fused matrix; the values stay
        m2 = before.clone()
        q2, k2 = (t.unflatten(-1, (-1, d)) for t in torch.split(m2, [hq * d, h * d, h * d + 8], dim=-1)[:2])
        got = vq.rotate(q2, k2, f, c, tree_mask=tm, interleaved=interleaved, scale=1.25, q_out=q2, k_out=k2)
        assert got[0] is q2 and torch.equal(q2, qo) and torch.equal(k2, ko)
        assert torch.equal(m2[..., (hq + h) * d:], before[..., (hq + h) * d:])


@pytest.mark.parametrize("at", [1 << 20, (1 << 24) - 1, 12345678])
def test_far_positions(at):
    """The angle's whole turns are dropped in 64 bits: at 2^24 an fp32 angle
    would be off by a radian."""
    m, q, k, _ = _fused(1, 5, 2, 2, 64, "f16", at % 97)
    freq = _freq(64, 10000.0)
    ctx = np.array([at], np.int32)
    qo, ko = vq.rotate(q, k, torch.from_numpy(freq).cuda(), torch.from_numpy(ctx).cuda())
    _check(qo, q, R.positions(ctx, None, 5), freq, False, 1.0, "f16")


def test_long_prompt():
    m, q, k, _ = _fused(2, 3001, 4, 1, 64, "bf16", 5)
    freq = _freq(32, 1e4, 8.0)
    ctx = np.array([17, 900], np.int32)
    qo, ko = vq.rotate(q, k, torch.from_numpy(freq).cuda(), torch.from_numpy(ctx).cuda(), interleaved=True)
    pos = R.positions(ctx, None, 3001)
    _check(qo, q, pos, freq, True, 1.0, "bf16")
    _check(ko, k, pos, freq, True, 1.0, "bf16")


def test_negative_lengths_and_infinities():
    """A negative length counts as 0; what one pair holds stays in that pair."""
    m, q, k, _ = _fused(1, 2, 2, 1, 64, "f16", 9)
    freq = _freq(64)
    f = torch.from_numpy(freq).cuda()
    a = vq.rotate(q, k, f, torch.tensor([-5], dtype=torch.int32, device="cuda"))
    b = vq.rotate(q, k, f, torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert torch.equal(a[0], b[0])
    q2 = q.clone()
    q2[0, 1, 1, 3] = float("inf")
    got, _ = vq.rotate(q2, k, f, torch.tensor([0], dtype=torch.int32, device="cuda"))
    changed = (got != b[0]).nonzero().tolist()
    assert [0, 1, 1, 3] in changed and all(c in ([0, 1, 1, 3], [0, 1, 1, 35]) for c in changed)


def test_captured_and_replayed():
    m, q, k, _ = _fused(2, 6, 8, 2, 128, "bf16", 3)
    f = torch.from_numpy(_freq(128)).cuda()
    c = torch.tensor([5, 70000], dtype=torch.int32, device="cuda")
    qo, ko = torch.empty(2, 6, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 6, 2, 128, dtype=torch.bfloat16, device="cuda")
    want = vq.rotate(q, k, f, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq.rotate(q, k, f, c, q_out=qo, k_out=ko)
    for _ in range(3):
        qo.zero_(), ko.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_binding_checks():
    m, q, k, _ = _fused(2, 6, 8, 2, 64, "bf16", 3)
    f = torch.from_numpy(_freq(64)).cuda()
    c = torch.zeros(2, dtype=torch.int32, device="cuda")
    big = torch.empty(2, 6, 800, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q_out=m[..., 64:576].unflatten(-1, (8, 64))), dict(k_out=m[..., :128].unflatten(-1, (2, 64))),
                dict(q_out=big[..., :512].unflatten(-1, (8, 64)), k_out=big[..., 504:632].unflatten(-1, (2, 64)))):
        with pytest.raises(ValueError, match="share"):
            vq.rotate(q, k, f, c, **bad)
    for bad in (dict(inv_freq=f.double()), dict(inv_freq=f[None]), dict(ctx_len=c.long()), dict(ctx_len=c[:1]),
                dict(tree_mask=torch.zeros(2, 5, dtype=torch.int64, device="cuda")), dict(q_out=torch.empty_like(q).half()),
                dict(q=q.float(), k=k.float()), dict(k=k[:1])):
        with pytest.raises((ValueError, TypeError, vq.VqError)):
            vq.rotate(**(dict(q=q, k=k, inv_freq=f, ctx_len=c) | bad))
    with pytest.raises(vq.VqError):
        vq.rotate(q, k, f[:4].contiguous(), c)


def test_offsets_past_32_bits():
    """Rows 8,000 elements apart in a fused matrix of 4.8 10^9 elements."""
    B, n, d = 3, 200000, 64
    m = torch.zeros(B, n, 8000, dtype=torch.float16, device="cuda")
    m[2, -1] = torch.randn(8000, generator=torch.Generator().manual_seed(1)).half().cuda()
    q, k = m[..., 7000:7064].unflatten(-1, (1, d)), m[..., 7872:8000].unflatten(-1, (2, d))
    freq = _freq(64)
    ctx = np.array([1, 2, 50], np.int32)
    qo, ko = vq.rotate(q, k, torch.from_numpy(freq).cuda(), torch.from_numpy(ctx).cuda())
    assert not qo[:2].any() and not ko[2, :-1].any()
    pos = np.array([[50 + n - 1]])
    _check(qo[2:, -1:], q[2:, -1:], pos, freq, False, 1.0, "f16")
    _check(ko[2:, -1:], k[2:, -1:], pos, freq, False, 1.0, "f16")
