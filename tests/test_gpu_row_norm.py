"""The residual update with its norms and the row quantizer against 64-bit
definitions."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _rows(n, c, dt, gen, size=1.0):
    x = size * torch.randn(n, c, generator=gen)
    x[:, c // 3] *= 40.0
    return x.to(DT[dt]).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _within(got, want, bound, out):
    worst = (np.abs(_np(got) - want) / R.rounded(want, bound, out)).max()
    assert worst <= 1.0, worst


CASES = [(1, 16, "f32"), (2, 48, "bf16"), (3, 512, "f16"), (5, 528, "f32"), (4, 1040, "bf16"), (1, 5120, "bf16"),
         (3, 8192, "f32"), (2, 8208, "f16"), (2, 16400, "bf16"), (2, 32768, "f32"), (300, 64, "bf16")]


@pytest.mark.parametrize("n,c,res", CASES)
@pytest.mark.parametrize("post,gate", [(False, None), (True, "channel"), (True, "row"), (False, "row")])
def test_residual_norm(n, c, res, post, gate):
    gen = torch.Generator().manual_seed(n + c)
    half = res if res != "f32" else ("bf16" if c % 32 else "f16")
    r, y = _rows(n, c, res, gen, 3.0), _rows(n, c, half, gen)
    w = (1 + 0.2 * torch.randn(c, generator=gen)).cuda()
    pw = (1 + 0.2 * torch.randn(c, generator=gen)).cuda() if post else None
    gt = None
    if gate == "channel":
        gt = torch.randn(c, generator=gen).cuda()
    elif gate == "row":
        gt = torch.rand(n, c, generator=gen).to(DT[half]).cuda()
    x, ex, h, eh = R.norm(_np(r), _np(y), _np(w), None if pw is None else _np(pw), None if gt is None else _np(gt),
                          float(np.float32(0.35)), float(np.float32(1e-5)))
    ro, out = torch.empty_like(r), torch.empty(n, c, dtype=DT[half], device="cuda")
    got = vq.residual_norm(r, y, w, post_weight=pw, gate=gt, alpha=0.35, eps=1e-5, out=out, residual_out=ro)
    assert got is out
    _within(ro, x, ex, res)
    _within(out, h, eh, half)
    # 8 bits: the scale from the largest, every code within half a step of its value
    q, s = vq.residual_norm(r, y, w, post_weight=pw, gate=gt, alpha=0.35, eps=1e-5,
                            out=torch.empty(n, c, dtype=torch.int8, device="cuda"),
                            scales_out=torch.empty(n, device="cuda"))
    top = np.abs(h).max(1)
    at = np.abs(h).argmax(1)
    assert (np.abs(_np(s) * 127 - top) <= eh.max(1) + 2 * R.U * top + eh[np.arange(n), at]).all()
    off = np.abs(_np(q) * _np(s)[:, None] - h)
    assert (off <= 0.5 * _np(s)[:, None] * (1 + 1e-5) + eh + 130 * 3 * R.U * _np(s)[:, None]).all()
    # in place
    same = r.clone()
    vq.residual_norm(same, y, w, post_weight=pw, gate=gt, alpha=0.35, eps=1e-5, out=out, residual_out=same)
    assert torch.equal(same, ro)


@pytest.mark.parametrize("n,c,res", CASES)
def test_norm_alone(n, c, res):
    gen = torch.Generator().manual_seed(c)
    r = _rows(n, c, res, gen)
    for w in (None, torch.randn(c, generator=gen).cuda()):
        for half in ("bf16", "f16"):
            out = torch.empty(n, c, dtype=DT[half], device="cuda")
            vq.residual_norm(r, weight=w, out=out)
            _, _, h, eh = R.norm(_np(r), None, None if w is None else _np(w), None, None, 1.0, float(np.float32(1e-6)))
            _within(out, h, eh, half)


def test_rows_of_zeros_and_without_eps():
    z = torch.zeros(3, 64, device="cuda")
    z[1] = 2.0
    out = torch.empty(3, 64, dtype=torch.float16, device="cuda")
    vq.residual_norm(z, out=out)
    assert (out[0] == 0).all() and (out[1] == 1).all() and (out[2] == 0).all()
    vq.residual_norm(z, out=out, eps=0.0)  # 0 / 0
    assert torch.isnan(out[0]).all() and (out[1] == 1).all()
    q, s = vq.residual_norm(z, out=torch.empty(3, 64, dtype=torch.int8, device="cuda"), scales_out=z[:, 0].clone())
    assert s.tolist()[0] == 0 and (q[0] == 0).all() and (q[1] == 127).all()


@pytest.mark.parametrize("n,k", [(1, 16), (3, 48), (2, 5120), (5, 8208), (2, 17408), (2, 32768), (700, 528)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_quantizer_bit_for_bit(n, k, dt):
    gen = torch.Generator().manual_seed(n * k)
    x = _rows(n, k, dt, gen)
    x[0, 5] = 0.0
    if n > 2:
        x[1] = 0.0
        x[2, :8] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 63.5], device="cuda").to(x.dtype)
        x[2, 8:] = 0.0
    q, s = vq.quant_rows_int8(x, torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda"))
    want_q, want_s = R.quant(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


def test_quantizer_extremes():
    """Infinities and NaN mark their row alone; the smallest numbers; a row at the type's largest."""
    x = torch.randn(7, 80, device="cuda")
    x[0, 3], x[1, 79], x[2, 0] = float("inf"), float("nan"), float("-inf")
    x[3] *= 1e-45
    x[4] *= 1e-38
    x[5] = 3.4e38
    q, s = vq.quant_rows_int8(x, torch.empty(7, 80, dtype=torch.int8, device="cuda"), torch.empty(7, device="cuda"))
    want_q, want_s = R.quant(x.cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True) and np.array_equal(q.cpu().numpy(), want_q)
    assert not q[:3].any() and torch.isnan(s[:3]).all() and not torch.isnan(s[3:]).any()


def test_many_rows():
    """A row's bits do not depend on the other rows."""
    gen = torch.Generator().manual_seed(3)
    r, y = _rows(5000, 144, "bf16", gen), _rows(5000, 144, "bf16", gen)
    w = torch.rand(144, generator=gen).cuda()
    a = vq.residual_norm(r, y, w, out=torch.empty_like(r), residual_out=torch.empty_like(r))
    for at in (0, 4999, 77):
        b = vq.residual_norm(r[at:at + 1], y[at:at + 1], w, out=torch.empty_like(r[:1]))
        assert torch.equal(a[at:at + 1], b)


def test_captured_and_replayed():
    gen = torch.Generator().manual_seed(4)
    r, y = _rows(9, 2064, "f16", gen), _rows(9, 2064, "f16", gen)
    q, s, ro = torch.empty(9, 2064, dtype=torch.int8, device="cuda"), torch.empty(9, device="cuda"), torch.empty_like(r)
    vq.residual_norm(r, y, out=q, scales_out=s, residual_out=ro)
    want = q.clone(), s.clone(), ro.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vq.residual_norm(r, y, out=q, scales_out=s, residual_out=ro)
    for _ in range(3):
        q.zero_(), s.zero_(), ro.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(s, want[1]) and torch.equal(ro, want[2])


def test_binding_checks():
    r = torch.randn(4, 64, device="cuda")
    y, w = r.half(), torch.ones(64, device="cuda")
    out, ro = torch.empty_like(y), torch.empty_like(r)
    with pytest.raises(ValueError, match="share"):
        vq.residual_norm(r, y, w, out=y, residual_out=ro)
    with pytest.raises(ValueError, match="share"):
        vq.residual_norm(r.view(-1)[:192].view(3, 64), y[:3], w, out=out[:3], residual_out=r.view(-1)[64:].view(3, 64))
    for bad in (dict(weight=w.half()), dict(gate=torch.ones(4, 64, device="cuda")), dict(gate=w[:32]),
                dict(residual_out=ro.half()), dict(y=y[:3]), dict(out=out[:, :32]), dict(y=y[:, ::2])):
        with pytest.raises((ValueError, TypeError)):
            vq.residual_norm(r, **(dict(y=y, weight=w, out=out, residual_out=ro) | bad))
    with pytest.raises(TypeError):
        vq.quant_rows_int8(r.double(), torch.empty(4, 64, dtype=torch.int8, device="cuda"), w[:4].clone())


def test_offsets_past_32_bits():
    n, c = 140000, 32768
    x = torch.zeros(n, c, dtype=torch.bfloat16, device="cuda")
    rows = [0, 65535, 131071, 131072, n - 1]
    gen = torch.Generator().manual_seed(8)
    for r in rows:
        x[r] = torch.randn(c, generator=gen).to(torch.bfloat16).cuda()
    q, s = vq.quant_rows_int8(x, torch.empty(n, c, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda"))
    want_q, want_s = R.quant(x[rows].float().cpu().numpy())
    assert np.array_equal(s[rows].cpu().numpy(), want_s) and np.array_equal(q[rows].cpu().numpy(), want_q)
    assert not q[1].any() and not q[n - 2].any()
    out = torch.empty_like(x)
    vq.residual_norm(x, out=out)
    _, _, h, eh = R.norm(_np(x[rows]), None, None, None, None, 1.0, float(np.float32(1e-6)))
    _within(out[rows], h, eh, "bf16")
