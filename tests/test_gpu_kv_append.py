"""Cache append on the GPU: copies, so every element has to be equal, and
every element that is not written has to stay as it was."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import tree_ref as R

pytestmark = pytest.mark.gpu


def _bits(g, *shape):
    return g.integers(0, 1 << 16, size=shape, dtype=np.uint16)  # NaN patterns too: only bits move


def _t(a, dtype=torch.bfloat16):
    return torch.from_numpy(a.view(np.int16).copy()).view(dtype).cuda()


def _np(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _check(seed, L, B, n, H, D, page, lens, path=None, count=None, layers_dim=True, pad=0, table=None, W=None,
           dtype=torch.bfloat16):
    g = np.random.Generator(np.random.PCG64(seed))
    need = [max(1, -(-(max(x, 0) + n) // page)) for x in lens]
    W = max(need) if W is None else W
    P = sum(need) + 2
    if table is None:
        pool = g.permutation(P)
        table, at = np.full((B, W), -1, np.int32), 0
        for b in range(B):
            c = min(W, need[b])
            table[b, :c] = pool[at:at + c]
            at += c
    kc, vc = _bits(g, L, P, H, page, D), _bits(g, L, P, H, page // 32, D, 32)
    k, v = _bits(g, L, B, n, H * D + pad), _bits(g, L, B, n, H * D + 2 * pad)
    kr, vr = (x[..., :H * D].reshape(L, B, n, H, D) for x in (k, v))
    lens = np.array(lens, np.int32)
    want_k, want_v, want_len = R.append(kr, vr, kc, vc, table, lens, path, count)
    dk, dv = (_t(x, dtype)[..., :H * D].unflatten(-1, (H, D)) for x in (k, v))
    ck, cv = _t(kc, dtype), _t(vc, dtype)
    dev = [None if x is None else torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
           for x in (table, lens, path, count)]
    if layers_dim:
        got = vq.kv_append(dk, dv, ck, cv, dev[0], dev[1], path=dev[2], count=dev[3])
    else:
        got = vq.kv_append(dk[0], dv[0], ck[0], cv[0], dev[0], dev[1], path=dev[2], count=dev[3])
    torch.cuda.synchronize()
    assert np.array_equal(_np(ck), want_k) and np.array_equal(_np(cv), want_v)
    assert got.cpu().numpy().tolist() == want_len.tolist()


@pytest.mark.parametrize("D,page", [(64, 32), (128, 64), (256, 256)])
@pytest.mark.parametrize("n,lens", [(1, [0]), (1, [31, 32, 33]), (7, [5, 0]), (33, [61, 3, 32]), (300, [0, 17])])
def test_rows_in_order(D, page, n, lens):
    _check(n + D, 1, len(lens), n, 2, D, page, lens, layers_dim=False)
    _check(n + D, 2, len(lens), n, 3, D, page, lens, pad=8, dtype=torch.float16)


def test_paths():
    g = np.random.Generator(np.random.PCG64(3))
    B, n = 6, 16
    path = np.full((B, n), -1, np.int32)
    count = np.array([0, 1, 5, 16, 9, 2], np.int32)
    for b in range(B):
        path[b, :count[b]] = np.sort(g.permutation(n)[:count[b]])
    _check(1, 3, B, n, 2, 128, 64, [0, 63, 60, 100, 31, 7], path=path, count=count)
    # rows in any order and repeated, out of range, negative and too large counts, a path without counts
    path = g.integers(-2, n + 2, size=(B, n)).astype(np.int32)
    _check(2, 2, B, n, 1, 64, 32, [0, 63, 60, 100, 31, 7], path=path, count=np.array([-3, 40, 16, 3, 1, 9], np.int32))
    _check(3, 2, B, n, 1, 64, 32, [0, 63, 60, 100, 31, 7], path=path)
    _check(4, 2, B, n, 1, 64, 32, [0, 63, 60, 100, 31, 7], count=count)


def test_what_does_not_fit_is_dropped():
    _check(5, 1, 3, 50, 2, 64, 32, [20, 64, 1000], W=2)
    _check(6, 2, 3, 9, 2, 64, 32, [-4, 30, 0], W=2)
    _check(7, 2, 2, 40, 2, 64, 32, [3, 30], table=np.array([[0, -1, 2], [1, 1 << 24, 3]], np.int32))


def test_what_was_appended_is_what_attention_reads():
    """Tokens appended in uneven runs, then attended to: the outputs of the
    same tokens given as nodes of a chain."""
    B, n, Hq, H, D, page = 2, 24, 4, 2, 128, 32
    gen = torch.Generator().manual_seed(11)
    q, k, v = (torch.randn(B, n, h, D, generator=gen).to(torch.float16).cuda() for h in (Hq, H, H))
    kc = torch.zeros(4, H, page, D, dtype=torch.float16, device="cuda")
    vc = torch.zeros(4, H, page // 32, D, 32, dtype=torch.float16, device="cuda")
    table = torch.tensor([[2, 1], [0, 3]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    whole = vq.tree_attention(q, k, v, kc, vc, table, zero)
    lens = zero
    at = 0
    for run in (1, 5, 2, 9, 6):
        lens = vq.kv_append(k[:, at:at + run].contiguous(), v[:, at:at + run].contiguous(), kc, vc, table, lens)
        at += run
    last = vq.tree_attention(q[:, at:].contiguous(), k[:, at:].contiguous(), v[:, at:].contiguous(), kc, vc, table, lens)
    torch.cuda.synchronize()
    assert lens.tolist() == [23, 23]
    # both round the probabilities and the output once: each within 2 * 2^-11 of |v| <= 5
    assert (whole[:, at:].float() - last.float()).abs().max().item() <= 4 * 2.0 ** -11 * 5
