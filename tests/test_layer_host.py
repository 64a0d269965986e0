"""The decoder-layer operators on the host: refused arguments (nothing is
enqueued), workspace sizes, and the 64-bit definitions against closed forms."""
import math

import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import layer_ref as R

# fake, 16-byte-aligned addresses: never dereferenced, validation fails first
P = [0x10000 * (i + 1) for i in range(16)]
BIG = 1 << 40
F32, BF16, F16, I8 = vq.DTYPE_F32, vq.DTYPE_BF16, vq.DTYPE_F16, vq.DTYPE_I8
ROOM = (1 << 24) + 16


def _gemm(w=P[0], ws=P[1], x=P[2], xs=P[3], bias=P[4], out=P[5], dt=BF16, n=3, m=32, k=64, wk=P[6], wb=BIG):
    return vq.lib().vq_gemm_w8a8(w, ws, x, xs, bias, out, dt, n, m, k, wk, wb, None)


def _gated(w=P[0], ws=P[1], u=P[7], us=P[8], x=P[2], xs=P[3], act=0, out=P[5], dt=BF16, n=3, m=32, k=64, wk=P[6],
           wb=BIG):
    return vq.lib().vq_gated_w8a8(w, ws, u, us, x, xs, act, out, dt, n, m, k, wk, wb, None)


@pytest.mark.parametrize("call,needed,matrices,vectors", [
    (_gemm, ("w", "ws", "x", "xs", "out"), ("w", "x", "out", "wk"), ("ws", "xs", "bias")),
    (_gated, ("w", "ws", "u", "us", "x", "xs", "out"), ("w", "u", "x", "out", "wk"), ("ws", "us", "xs"))])
def test_product_refusals(call, needed, matrices, vectors):
    for name in needed:
        assert call(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    for name in matrices:
        assert call(**{name: 0x10008}) == vq.VQ_ERR_MISALIGNED, name
    for name in vectors:
        assert call(**{name: 0x10002}) == vq.VQ_ERR_MISALIGNED, name
    for dt in (I8, 0, 9):
        assert call(dt=dt) == vq.VQ_ERR_BAD_DTYPE
    for bad in (dict(n=0), dict(n=-1), dict(n=ROOM), dict(m=0), dict(m=ROOM), dict(k=0), dict(k=8), dict(k=72),
                dict(k=131072), dict(k=-16)):
        assert call(**bad) == vq.VQ_ERR_BAD_SHAPE, bad
    if not torch.cuda.is_available():  # past the checks
        for ok in ({}, dict(ws=0x10004), dict(wk=None, wb=0), dict(k=131056), dict(k=16, m=1, n=1)):
            assert call(**ok) == vq.VQ_ERR_DEVICE, ok


def test_gated_activation():
    assert _gated(act=3) == vq.VQ_ERR_BAD_CONFIG and _gated(act=-1) == vq.VQ_ERR_BAD_CONFIG


def test_product_workspace_sizes():
    sizes = [vq.w8a8_workspace_bytes(n) for n in (1, 16, 17, 64, 65, 300, 1 << 24)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    for n in (0, -1, ROOM):
        assert vq.w8a8_workspace_bytes(n) == 0


def _norm(r=P[0], rdt=F32, y=P[1], ydt=BF16, post=P[2], gate=P[3], rows=0, alpha=1.0, w=P[4], eps=1e-6, ro=P[5],
          out=P[6], odt=I8, so=P[7], n=3, c=64):
    return vq.lib().vq_residual_norm(r, rdt, y, ydt, post, gate, rows, alpha, w, eps, ro, out, odt, so, n, c, None)


def test_norm_refusals():
    for name in ("r", "out", "so"):
        assert _norm(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    for name in ("r", "y", "post", "gate", "w", "ro", "out"):
        assert _norm(**{name: 0x10008}) == vq.VQ_ERR_MISALIGNED, name
    assert _norm(so=0x10002) == vq.VQ_ERR_MISALIGNED
    for bad in (dict(rdt=I8), dict(ydt=F32), dict(odt=F32, so=None), dict(odt=BF16), dict(odt=0, so=None)):
        assert _norm(**bad) == vq.VQ_ERR_BAD_DTYPE, bad
    for bad in (dict(n=0), dict(n=ROOM), dict(c=0), dict(c=8), dict(c=40), dict(c=32784)):
        assert _norm(**bad) == vq.VQ_ERR_BAD_SHAPE, bad
    for bad in (dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(y=None),
                dict(y=None, gate=None, ro=None), dict(y=None, post=None, ro=None),
                dict(y=None, post=None, gate=None)):
        assert _norm(**bad) == vq.VQ_ERR_BAD_CONFIG, bad


def _quant(x=P[0], dt=BF16, q=P[1], s=P[2], n=3, k=64):
    return vq.lib().vq_quant_rows_int8(x, dt, q, s, n, k, None)


def test_quant_refusals():
    for name in ("x", "q", "s"):
        assert _quant(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    assert _quant(x=0x10004) == _quant(q=0x10008) == _quant(s=0x10001) == vq.VQ_ERR_MISALIGNED
    assert _quant(dt=I8) == vq.VQ_ERR_BAD_DTYPE
    for bad in (dict(n=0), dict(n=ROOM), dict(k=0), dict(k=24), dict(k=32784)):
        assert _quant(**bad) == vq.VQ_ERR_BAD_SHAPE, bad


def _rotate(q=P[0], qs=512, k=P[1], ks=128, dt=BF16, f=P[2], ctx=P[3], mask=P[4], qo=P[5], qos=512, ko=P[6], kos=128,
            b=2, n=4, hq=8, h=2, d=64, rot=64, il=0):
    return vq.lib().vq_rotate(q, qs, k, ks, dt, f, ctx, mask, qo, qos, ko, kos, b, n, hq, h, d, rot, il, 1.0, None)


def test_rotate_refusals():
    for name in ("q", "f", "ctx", "qo", "k", "ko"):
        assert _rotate(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    for name in ("q", "k", "qo", "ko"):
        assert _rotate(**{name: 0x10008}) == vq.VQ_ERR_MISALIGNED, name
    assert _rotate(mask=0x10004) == _rotate(f=0x10002) == _rotate(ctx=0x10001) == vq.VQ_ERR_MISALIGNED
    for dt in (F32, I8, 0):
        assert _rotate(dt=dt) == vq.VQ_ERR_BAD_DTYPE
    for bad in (dict(b=0), dict(n=0), dict(n=65), dict(b=1 << 20, n=9, mask=None), dict(b=ROOM, n=1), dict(hq=0),
                dict(hq=1025), dict(h=0), dict(h=1025), dict(d=72), dict(d=528, qs=8 * 528, qos=8 * 528), dict(rot=0),
                dict(rot=8), dict(rot=72), dict(rot=80), dict(qs=504), dict(qs=516), dict(ks=120), dict(qos=508),
                dict(kos=64), dict(qs=ROOM)):
        assert _rotate(**bad) == vq.VQ_ERR_BAD_SHAPE, bad
    if not torch.cuda.is_available():
        for ok in ({}, dict(k=None, ko=None, h=0, ks=0, kos=0), dict(n=65, mask=None), dict(rot=16), dict(mask=0x10008)):
            assert _rotate(**ok) == vq.VQ_ERR_DEVICE, ok


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a device every valid call is refused")
def test_no_device_is_an_error():
    assert _gemm() == _gated() == _norm() == _quant() == _rotate() == vq.VQ_ERR_DEVICE


def test_binding_refusals():
    i8, f = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    out = torch.zeros(4, 4, dtype=torch.float16)
    for call in (lambda: vq.gemm_w8a8(i8, f, i8, f, torch.zeros(4, 5)),
                 lambda: vq.gemm_w8a8(i8, f, i8[0], f, out),
                 lambda: vq.gated_w8a8(i8, f, i8, f, i8, f, torch.zeros(3, 4)),
                 lambda: vq.gated_w8a8(i8, f, i8, f, i8, f, out, activation="relu"),
                 lambda: vq.residual_norm(out[0], out=out),
                 lambda: vq.residual_norm(out, out=i8),
                 lambda: vq.residual_norm(out, out=out, scales_out=f),
                 lambda: vq.residual_norm(out, out=out, gate=f),
                 lambda: vq.residual_norm(out, out=out, residual_out=out),
                 lambda: vq.quant_rows_int8(out[0], i8, f),
                 lambda: vq.rotate(out, None, f, f)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError, match="y must"):
        vq.residual_norm(out, torch.zeros(4, 4), out=out)
    q = torch.zeros(1, 2, 4, 16, dtype=torch.float16)
    with pytest.raises(TypeError, match="one dtype"):
        vq.rotate(q, q.bfloat16(), f, f)


def test_devices():
    class T:
        def __init__(self, dev):
            self.get_device = lambda: dev
    a = vq._Args()
    with pytest.raises(ValueError, match="x must be a device tensor"):
        a.on(T(-1), "x")
    a.on(T(1), "x"), a.on(T(1), "y")
    for dev in (-1, 0, 2):
        with pytest.raises(ValueError, match="z must"):
            a.on(T(dev), "z")


def test_shared_memory_is_seen():
    t = torch.zeros(8, 64)
    assert vq._span(t[2:4]) == (t.data_ptr() + 512, t.data_ptr() + 1024)
    a = vq._Args()
    a.here = lambda: None

    def ranges(*parts):
        a.ranges = [(p.data_ptr(), p.data_ptr() + p.nbytes, name) for name, p in parts]
    ranges(("x", t[3:]), ("out", t[2:4]))
    with pytest.raises(ValueError, match="out must not share memory with x"):
        a.apart(1)
    ranges(("x", t[4:]), ("y", t[:2]), ("out", t[2:4]))
    a.apart(1)
    ranges(("x", t[:2]), ("y", t[2:4]), ("out", t[2:4]))
    a.apart(1, ("out", "y"))
    with pytest.raises(ValueError, match="share"):
        a.apart(1, ("out", "x"))
    ranges(("x", t[1:3]), ("out", t[2:4]))
    with pytest.raises(ValueError, match="share"):
        a.apart(1, ("out", "x"))
    ranges(("x", t[4:]), ("one", t[:2]), ("two", t[1:4]))
    with pytest.raises(ValueError, match="two must not share memory with one"):
        a.apart(2)
    fused = torch.zeros(6, 96)
    a, b = fused[:, :64], fused[:, 64:]
    assert not vq._share_rows(a, 96, 64, b, 96, 32) and not vq._share_rows(b, 96, 32, a, 96, 64)
    assert not vq._share_rows(fused[1:, :64], 96, 64, fused[:-1, 64:], 96, 32)
    assert vq._share_rows(a, 96, 64, fused[:, 48:], 96, 48) and vq._share_rows(fused[:, 48:], 96, 48, a, 96, 64)
    assert vq._share_rows(a, 96, 64, fused[1:, :64], 96, 64) and vq._share_rows(a, 96, 64, fused.view(12, 48), 48, 32)


def test_definition_of_the_products():
    g = np.random.Generator(np.random.PCG64(1))
    x, w = (g.integers(-128, 128, (3, 32)).astype(np.int8) for _ in range(2))
    y, err = R.product(x, np.ones(3), w, np.full(3, 0.5), np.array([0.0, 1.0, 2.0]))
    for i in range(3):
        for j in range(3):
            assert y[i, j] == 0.5 * sum(int(a) * int(b) for a, b in zip(x[i], w[j])) + j
    for kind, at in (("silu", lambda v: v / (1 + math.exp(-v))), ("gelu", lambda v: v * 0.5 * (1 + math.erf(v / 2 ** 0.5))),
                     ("gelu_tanh", lambda v: 0.5 * v * (1 + math.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))))):
        for v in (-3.0, -0.5, 0.0, 0.7, 4.0):
            assert abs(R.activate(np.array([v]), 0.0, kind)[0][0] - at(v)) < 1e-12


def test_definition_of_the_norm():
    r = np.array([[3.0, -4.0, 0.0, 0.0]])
    x, _, h, _ = R.norm(r, None, np.array([1.0, 2, 1, 1]), None, None, 1.0, 0.0)
    assert np.allclose(h, [[1.2, -3.2, 0, 0]]) and (x == r).all()
    x, _, h, _ = R.norm(r, np.array([[2.0, 0, 0, 0]]), None, np.array([5.0, 1, 1, 1]), np.array([0.5, 1, 1, 1]), 0.2, 0.0)
    assert np.allclose(x, [[3 + 0.2 * 0.5 * 5 * 2, -4, 0, 0]])


def test_definition_of_the_quantizer():
    q, s = R.quant(np.array([[1.0, -2.0, 0.5, 0.0], [0, 0, 0, 0], [np.inf, 1, 1, 1], [np.nan, 1, 1, 1]], np.float32))
    assert q[0].tolist() == [64, -127, 32, 0] and not q[1:].any()
    assert s[0] == np.float32(2) / np.float32(127) and s[1] == 0 and np.isnan(s[2:]).all()


def test_definition_of_the_rotation():
    """A quarter turn swaps a pair, a full turn keeps it; depths come from the ancestors' bits."""
    t = np.arange(16.0).reshape(1, 1, 1, 16)
    freq = np.array([math.pi / 2, 2 * math.pi])
    out, _ = R.rotate(t, np.array([[1]]), freq, False, 1.0)
    assert np.allclose(out[0, 0, 0, :4], [-2, 1, 0, 3]) and (out[..., 4:] == t[..., 4:]).all()
    out, _ = R.rotate(t, np.array([[1]]), freq, True, 2.0)
    assert np.allclose(out[0, 0, 0, :4], [-2, 0, 4, 6])
    masks = np.array([[1, 3, 5, 11]], np.uint64)
    assert R.positions([7], masks, 4).tolist() == [[7, 8, 8, 9]] and R.positions([-3], None, 2).tolist() == [[0, 1]]
