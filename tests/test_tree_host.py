"""The speculative-step operators on the host: refused arguments (nothing is
enqueued), workspace sizes, and the 64-bit reference against closed forms."""
import math

import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import tree_ref as R

# fake, 16-byte-aligned addresses: never dereferenced, validation fails first
P = [0x10000 * (i + 1) for i in range(16)]
BIG = 1 << 40


def _attn(q=P[0], qs=1024, k=P[1], ks=256, v=P[2], vs=256, dt=vq.DTYPE_BF16, kc=P[3], vc=P[4], table=P[5], ctx=P[6],
          mask=P[7], nodes=P[8], out=P[9], b=2, n=4, hq=8, h=2, d=128, page=64, pages=10, w=4, ws=P[10], wsb=BIG):
    return vq.lib().vq_tree_attention(q, qs, k, ks, v, vs, dt, kc, vc, table, ctx, mask, nodes, out, b, n, hq, h, d,
                                      page, pages, w, 0.1, ws, wsb, None)


def test_attention_refusals():
    for name in ("q", "k", "v", "kc", "vc", "table", "ctx", "out"):
        assert _attn(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    for name in ("q", "k", "v", "kc", "vc", "table", "ctx", "mask", "nodes", "out", "ws"):
        assert _attn(**{name: 0x10008}) == vq.VQ_ERR_MISALIGNED, name
    for dt in (vq.DTYPE_F32, vq.DTYPE_I8, 0):
        assert _attn(dt=dt) == vq.VQ_ERR_BAD_DTYPE
    for bad in (dict(b=0), dict(b=4097), dict(n=0), dict(n=65), dict(hq=7), dict(hq=0), dict(h=0), dict(h=3),
                dict(hq=1026, h=2), dict(d=96), dict(d=512), dict(page=48), dict(page=16), dict(page=512),
                dict(pages=0), dict(w=0), dict(w=(1 << 24) + 1), dict(w=-1), dict(qs=1020), dict(qs=1016), dict(ks=248),
                dict(vs=257), dict(vs=(1 << 24) + 8), dict(n=-1)):
        assert _attn(**bad) == vq.VQ_ERR_BAD_SHAPE, bad
    assert _attn(ws=None) == vq.VQ_ERR_WORKSPACE
    need = vq.tree_attention_workspace_bytes(2, 4, 8, 2, 128)
    assert need > 0 and _attn(wsb=need - 1) == vq.VQ_ERR_WORKSPACE
    assert vq.tree_attention_workspace_bytes(2, 65, 8, 2, 128) == 0
    assert vq.tree_attention_workspace_bytes(2, 4, 8, 3, 128) == 0


def _verify(t=P[0], d=P[1], dt=vq.DTYPE_BF16, tok=P[2], par=P[3], nodes=P[4], temp=P[5], u=P[6], e=P[7], o=P[8],
            path=P[9], cnt=P[10], b=2, n=4, vocab=1000, ws=P[11], wsb=BIG):
    return vq.lib().vq_tree_verify(t, d, dt, tok, par, nodes, temp, u, e, o, path, cnt, b, n, vocab, ws, wsb, None)


def test_verify_refusals():
    for name in ("t", "tok", "u", "e", "o", "path", "cnt"):
        assert _verify(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    for name in ("t", "d", "tok", "par", "nodes", "temp", "u", "e", "o", "path", "cnt", "ws"):
        assert _verify(**{name: 0x10004}) == vq.VQ_ERR_MISALIGNED, name
    assert _verify(dt=vq.DTYPE_I8) == vq.VQ_ERR_BAD_DTYPE
    for bad in (dict(b=0), dict(b=4097), dict(n=0), dict(n=65), dict(vocab=0), dict(vocab=(1 << 24) + 1)):
        assert _verify(**bad) == vq.VQ_ERR_BAD_SHAPE, bad
    need = vq.tree_verify_workspace_bytes(2, 4, 1000)
    assert need > 0 and _verify(wsb=need - 1) == vq.VQ_ERR_WORKSPACE and _verify(ws=None) == vq.VQ_ERR_WORKSPACE
    assert vq.tree_verify_workspace_bytes(2, 65, 1000) == 0


def _append(k=P[0], ks=256, v=P[1], vs=256, dt=vq.DTYPE_F16, kc=P[2], vc=P[3], table=P[4], ctx=P[5], path=P[6],
            cnt=P[7], ln=P[8], layers=3, b=2, n=4, h=2, d=128, page=64, pages=10, w=4):
    return vq.lib().vq_kv_append(k, ks, v, vs, dt, kc, vc, table, ctx, path, cnt, ln, layers, b, n, h, d, page, pages,
                                 w, None)


def test_append_refusals():
    for name in ("k", "v", "kc", "vc", "table", "ctx"):
        assert _append(**{name: None}) == vq.VQ_ERR_NULL_POINTER, name
    for name in ("k", "v", "kc", "vc", "table", "ctx", "path", "cnt", "ln"):
        assert _append(**{name: 0x10002}) == vq.VQ_ERR_MISALIGNED, name
    assert _append(dt=vq.DTYPE_F32) == vq.VQ_ERR_BAD_DTYPE
    for bad in (dict(layers=0), dict(layers=1025), dict(b=0), dict(n=0), dict(n=(1 << 24) + 1), dict(h=0), dict(d=80),
                dict(page=33), dict(pages=0), dict(w=0), dict(ks=255), dict(vs=128),
                dict(layers=1024, b=4096, n=1 << 20, h=2)):
        assert _append(**bad) == vq.VQ_ERR_BAD_SHAPE, bad


def test_append_refuses_what_no_launch_holds():
    """A thread writes 8 positions x 8 channels, and a grid dimension holds
    2^32 - 1 threads: more is refused as a size, before anything is enqueued."""
    for ok, sizes in ((True, dict(layers=1024, b=4096, n=1, h=15, d=128)), (False, dict(layers=1024, b=4096, n=1, h=16, d=128)),
                      (False, dict(layers=1024, b=4096, n=1, h=64, d=128)), (False, dict(layers=1, b=64, n=1 << 24, h=4, d=64)),
                      (True, dict(layers=1, b=63, n=1 << 24, h=4, d=64)), (False, dict(layers=1024, b=2048, n=33, h=16, d=128))):
        blocks = (sizes["n"] + 30) // 32 + 1
        threads = sizes["layers"] * sizes["b"] * blocks * sizes["h"] * sizes["d"] // 2
        assert (threads < 1 << 32) == ok
        if not ok:
            width = sizes["h"] * sizes["d"]
            assert _append(ks=width, vs=width, **sizes) == vq.VQ_ERR_BAD_SHAPE, sizes
        elif not torch.cuda.is_available():  # past the size checks
            assert _append(ks=sizes["h"] * sizes["d"], vs=sizes["h"] * sizes["d"], **sizes) == vq.VQ_ERR_DEVICE, sizes


@pytest.mark.skipif(torch.cuda.is_available(), reason="without a device every valid call is refused")
def test_no_device_is_an_error():
    assert _attn() == vq.VQ_ERR_DEVICE and _verify() == vq.VQ_ERR_DEVICE and _append() == vq.VQ_ERR_DEVICE


def test_binding_refusals():
    q = torch.zeros(2, 3, 4, 64, dtype=torch.float16)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.float16)
    kc, vc = torch.zeros(5, 2, 32, 64, dtype=torch.float16), torch.zeros(5, 2, 1, 64, 32, dtype=torch.float16)
    table, ctx = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        vq.tree_attention(q, k, k, kc, vc, table, ctx)
    with pytest.raises(ValueError, match="v_cache"):
        vq.tree_attention(q, k, k, kc, kc, table, ctx)
    with pytest.raises(TypeError, match="dtype"):
        vq.tree_attention(q.bfloat16(), k, k, kc, vc, table, ctx)
    with pytest.raises(ValueError, match="head_dim"):
        vq.tree_attention(torch.zeros(2, 3, 4, 128, dtype=torch.float16), k, k, kc, vc, table, ctx)
    with pytest.raises(ValueError, match="device"):
        vq.kv_append(k, k, kc, vc, table, ctx)
    with pytest.raises(ValueError, match="k_cache"):
        vq.kv_append(k[None], k[None], kc, vc, table, ctx)
    with pytest.raises(ValueError, match="draft"):
        vq._array(torch.zeros(2, 3, 8), "draft", (2, 3, 7), torch.float32)


def test_row_strides():
    class T:  # a tensor of this shape and strides on a device
        def __init__(self, t):
            self.shape, self.is_cuda, self.stride, self.is_contiguous = t.shape, True, t.stride, t.is_contiguous
    fused = torch.zeros(3, 5, 100 * 8)
    assert vq._rows(T(fused[..., 64:192].unflatten(-1, (2, 64))), "k", (3, 5, 2, 64)) == 800
    assert vq._rows(T(fused[:, :1, :128].unflatten(-1, (2, 64))), "k", (3, 1, 2, 64)) == 4000
    assert vq._rows(T(fused[:1, :1, :128].unflatten(-1, (2, 64))), "k", (1, 1, 2, 64)) == 128
    with pytest.raises(ValueError, match="evenly"):
        vq._rows(T(fused[:, :4, :128].unflatten(-1, (2, 64))), "k", (3, 4, 2, 64))
    with pytest.raises(ValueError, match="contiguous"):
        vq._rows(T(fused[..., :128].unflatten(-1, (64, 2)).transpose(-1, -2)), "k", (3, 5, 2, 64))


@pytest.mark.parametrize("base,shape", [
    ((3, 1, 2, 64), (3, 5, 2, 64)), ((1, 1, 2, 64), (3, 5, 2, 64)), ((1, 5, 2, 64), (3, 5, 2, 64)),
    ((1, 1, 2, 64), (1, 5, 2, 64)), ((1, 1, 2, 64), (3, 1, 2, 64)), ((3, 5, 1, 64), (3, 5, 2, 64)),
    ((3, 5, 2, 1), (3, 5, 2, 64)), ((4, 3, 1, 2, 64), (4, 3, 5, 2, 64)), ((4, 1, 5, 2, 64), (4, 3, 5, 2, 64)),
    ((1, 3, 5, 2, 64), (4, 3, 5, 2, 64))])
def test_expanded_rows_are_refused(base, shape):
    """A broadcast dimension has stride 0: no single row stride reaches every
    row, and one taken from the next dimension would lead past the storage."""
    t = torch.zeros(base).expand(shape)

    class T:
        is_cuda, stride, is_contiguous = True, t.stride, t.is_contiguous
    T.shape = t.shape
    with pytest.raises(ValueError, match="rows must|contiguous"):
        vq._rows(T(), "k", shape)


def test_overlapping_rows_are_refused():
    t = torch.zeros(4096).as_strided((3, 5, 2, 64), (5 * 64, 64, 64, 1))  # rows of 128, 64 apart

    class T:
        is_cuda, shape, stride, is_contiguous = True, t.shape, t.stride, t.is_contiguous
    with pytest.raises(ValueError, match="share"):
        vq._rows(T(), "k", (3, 5, 2, 64))


def test_reference_attention():
    """Equal scores average the values; a one-hot score picks one; the mask is obeyed."""
    g = np.random.Generator(np.random.PCG64(1))
    D, page = 4, 32
    kc, vc = np.zeros((3, 1, page, D)), g.standard_normal((3, 1, 1, D, page))
    table = np.array([[2, 0]], np.int32)
    q, k, v = np.zeros((1, 2, 1, D)), np.zeros((1, 2, 1, D)), g.standard_normal((1, 2, 1, D))
    out, _ = R.attention(q, k, v, kc, vc, table, [40], None, None, 0.5, "f16")
    past = np.concatenate([vc[2, 0, 0].T, vc[0, 0, 0].T[:8]])
    assert np.allclose(out[0, 0, 0], np.concatenate([past, v[0, :1, 0]]).mean(0))
    assert np.allclose(out[0, 1, 0], np.concatenate([past, v[0, :2, 0]]).mean(0))
    masks = np.array([[2, 0]], np.uint64)
    out, _ = R.attention(q, k, v, kc, vc, table, [0], masks, None, 0.5, "f16")
    assert np.allclose(out[0, 0, 0], v[0, 1, 0]) and (out[0, 1] == 0).all()
    q[..., 0] = 1000.0
    kc[0, 0, 3, 0] = 1.0
    out, _ = R.attention(q, k, v, kc, vc, table, [40], None, None, 0.5, "f16")
    assert np.allclose(out[0, 0, 0], vc[0, 0, 0, :, 3])


def test_reference_verify():
    """Two tokens by hand, p = (0.75, 0.25), q = (0.25, 0.75): token 1 is
    accepted below u = 1/3, token 0 always; after a rejection only token 0 has
    anything left."""
    ln3 = math.log(3.0)
    target, draft = np.array([[[ln3, 0.0]] * 3]), np.array([[[0.0, ln3]] * 3])
    e = np.ones((1, 2))

    def go(tokens, u, d=draft, parents=None):
        t, p, c, _ = R.verify(target, d, np.array([tokens]), parents, None, None, np.array([u]), e)
        return t[0].tolist(), p[0].tolist(), int(c[0])
    assert go([9, 1, 1], [0, 0.33, 0.34]) == ([1, 0, -1], [0, 1, -1], 2)
    assert go([9, 0, 1], [0, 0.99, 0.3]) == ([0, 1, 0], [0, 1, 2], 3)
    star = np.array([[-1, 0, 0]])
    # after rejecting token 1, r = (0.5, 0): a second child with token 0 is always accepted, token 1 never
    assert go([9, 1, 0], [0, 0.5, 0.99], parents=star) == ([0, 0, -1], [0, 2, -1], 2)
    assert go([9, 1, 1], [0, 0.5, 0.0], parents=star) == ([0, -1, -1], [0, -1, -1], 1)
    # given children: token 1 is accepted below its own probability
    assert go([9, 1, 0], [0, 0.24, 0.5], None, star)[2] == 2
    assert go([9, 1, 0], [0, 0.26, 0.99], None, star) == ([0, 0, -1], [0, 2, -1], 2)


def test_remainder_identity():
    """Nested differences and the one-scalar form of the remainder agree."""
    g = np.random.Generator(np.random.PCG64(2))
    p, q = (R.softmax(g.standard_normal(50)) for _ in range(2))
    left, S, s = p, 0.0, 1.0
    for _ in range(5):
        left = np.maximum(0, left / left.sum() - q) * s if S else np.maximum(0, p - q)
        S += s
        assert np.allclose(left, np.maximum(0, p - S * q))
        s = left.sum()
