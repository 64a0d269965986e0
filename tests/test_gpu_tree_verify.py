"""Acceptance of drafted trees on the GPU against the definition at 64 bits.

The results are whole numbers, so they have to be equal wherever no decision
on the way is a near tie: a decision compares two products of fp32 softmax
terms, each within about 1e-5 of its value (the exponent's rounding, |l / T| <=
30 times 2^-23, and the sums'), the remainders of close p and q several times
that; sequences with a decision nearer than 1e-3 (relative) are left out, and
most have to remain."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import tree_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NEAR = 1e-3


def _inputs(seed, B, n, V, dtype, drawn, branch=3, temps=(0.5, 1.0, 1.7), spread=2.0, near=0.7):
    g = np.random.Generator(np.random.PCG64(seed))
    tgt = torch.from_numpy((spread * g.standard_exponential((B, n, V))).astype(np.float32)).to(DT[dtype])
    drf = (tgt.float() + torch.from_numpy((near * g.standard_normal((B, n, V))).astype(np.float32))).to(DT[dtype])
    parents = R.random_trees(B, n, g, branch)
    temp = np.array([temps[b % len(temps)] for b in range(B)], np.float32)
    tok = np.zeros((B, n), np.int32)
    d = drf.to(torch.float64).numpy()
    for b in range(B):
        for i in range(1, n):
            row = d[b, parents[b, i]]
            if drawn:
                t = temp[b] if temp[b] > 0 else 1.0
                tok[b, i] = np.argmax(row / t - np.log(g.standard_exponential(V)))
            else:
                tok[b, i] = np.argsort(-row)[min(V - 1, i % branch)]
    return dict(target=tgt, draft=drf if drawn else None, tokens=tok, parents=parents,
                n_nodes=None, temperature=temp, uniforms=g.random((B, n), dtype=np.float32),
                noise=g.standard_exponential((B, V)).astype(np.float32) + np.float32(1e-12))


def _dev(x):
    return None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))).cuda()


def _run(c, **kw):
    out = vq.tree_verify(_dev(c["target"]), _dev(c["draft"]), _dev(c["tokens"]), _dev(c["uniforms"]), _dev(c["noise"]),
                         parents=_dev(c["parents"]), n_nodes=_dev(c["n_nodes"]), temperature=_dev(c["temperature"]),
                         **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy().astype(np.int64) for t in out]


def _check(c, got=None, keep_most=0.8):
    got = _run(c) if got is None else got
    f64 = [None if c[k] is None else c[k].to(torch.float64).numpy() for k in ("target", "draft")]
    tokens, path, count, margin = R.verify(*f64, c["tokens"], c["parents"], c["n_nodes"], c["temperature"],
                                           c["uniforms"], c["noise"])
    clear = margin > NEAR
    assert clear.mean() >= keep_most, clear.mean()
    for x, y in zip(got, (tokens, path, count)):
        assert np.array_equal(x[clear], y[clear])
    return count


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,n,V,branch", [(1, 1, 1, 1), (3, 2, 7, 1), (40, 16, 301, 3), (9, 64, 1000, 6),
                                          (4, 8, 5001, 1), (3, 12, 33000, 4)])
def test_trees(dtype, drawn, B, n, V, branch):
    _check(_inputs(3 + B + n + V, B, n, V, dtype, drawn, branch), keep_most=0.6)


@pytest.mark.parametrize("drawn", [True, False])
def test_chain_and_ragged(drawn):
    c = _inputs(20, 50, 9, 513, "bf16", drawn, branch=1)
    c["parents"] = None
    c["n_nodes"] = np.array([b % 11 for b in range(50)], np.int32)  # 0 and past n among them
    got = _run(c)
    _check(c, got)
    assert (got[2][::11] == 0).all() and (got[0][::11] == -1).all() and (got[1][::11] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_greedy_sequences_in_the_batch(dtype):
    c = _inputs(21, 30, 12, 400, dtype, True, temps=(0.0, 0.8))
    for b in range(0, 30, 2):  # drafted tokens that are often the greedy choice
        best = c["target"][b].float().numpy().argmax(-1)
        c["tokens"][b, 1:] = np.where(np.arange(1, 12) % 4 != 0, best[c["parents"][b, 1:]], 0)
    c["target"][0, 0, 17] = float("nan")
    c["target"][2, 0] = 1.0  # all tied: index 0
    c["target"][4, 0] = float("-inf")
    got = _run(c)
    count = _check(c, got)
    assert count[::2].max() > 2
    # a chain's greedy acceptance is vq_greedy_verify's
    c = _inputs(22, 4, 10, 999, dtype, True, branch=1, temps=(0.0,))
    c["tokens"][:, 1:] = c["target"][:, :-1].float().numpy().argmax(-1)
    c["tokens"][1, 6] = -1
    tokens, path, count = _run(c)
    for b in range(4):
        t, k = vq.greedy_verify(_dev(c["target"][b]), _dev(c["tokens"][b, 1:].copy()))
        k = int(k.item())
        assert k == count[b] and t.cpu().numpy()[:k].tolist() == tokens[b, :k].tolist()


def test_no_temperature_is_one():
    c = _inputs(23, 6, 5, 300, "f32", True, temps=(1.0,))
    want = _run(c)
    c["temperature"] = None
    for x, y in zip(_run(c), want):
        assert np.array_equal(x, y)


def test_tokens_and_parents_out_of_range():
    """Tokens outside the vocabulary are rejected; parents outside [0, i) drop the node."""
    for drawn in (True, False):
        c = _inputs(24, 60, 10, 97, "f32", drawn)
        c["tokens"][:, 3] = 97
        c["tokens"][:, 5] = -1
        c["tokens"][::2, 7] = 1 << 30
        c["parents"][:, 4] = [(-1, 4, 9, 1 << 20, -(1 << 31))[b % 5] for b in range(60)]
        _check(c)


def test_masked_tokens_and_equal_rows():
    """-inf logits (probability 0), p = q, and a drafter that is sure."""
    c = _inputs(25, 40, 8, 128, "f32", True)
    c["target"][:, :, 5::2] = float("-inf")
    c["draft"][::2, :, 3::2] = float("-inf")
    _check(c)
    c = _inputs(26, 40, 8, 128, "f32", True)
    c["draft"] = c["target"].clone()
    assert (_run(c)[2] > 1).mean() > 0.95  # p = q: every first child is accepted (u < 1)
    c = _inputs(27, 8, 4, 128, "f32", True)
    c["target"][:] = float("-inf")
    c["target"][:, :, 9] = 0.0
    c["draft"][:] = c["target"]
    c["tokens"][:] = 9
    tokens, path, count = _run(c)
    assert (count >= 2).all() and (tokens[:, 0] == 9).all()


def test_nothing_left_falls_back_to_the_target():
    """Every token of the target given and rejected: p stands in."""
    c = _inputs(28, 6, 4, 3, "f32", False)
    c["parents"][:] = np.array([-1, 0, 0, 0], np.int32)
    c["tokens"][:] = np.array([0, 0, 1, 2], np.int32)
    c["target"][:] = float("-inf")
    c["target"][:, :, 1] = 0.0                      # p is 1 at token 1
    c["tokens"][:, 2] = 0                           # and token 1 is not drafted
    c["tokens"][:, 3] = 2
    tokens, path, count = _run(c)
    assert (count == 1).all() and (tokens[:, 0] == 1).all()
    d = _inputs(29, 30, 5, 64, "f32", True)         # p = q and no child that could be accepted: p - q is 0
    d["draft"], d["tokens"][:] = d["target"].clone(), -1
    _check(d)
    c["tokens"][:, 1] = 1                           # drafted: accepted, since u < 1
    tokens, path, count = _run(c)
    assert (count == 2).all() and (tokens[:, 0] == 1).all()


@pytest.mark.parametrize("drawn", [True, False])
def test_first_token_follows_the_target(drawn):
    """Over many independent random numbers the first committed token has the
    target's distribution, whatever the drafter proposes: 3 x 4096 draws
    against p, chi-square with 11 degrees of freedom, 99.99% quantile 37.4."""
    V, n, B = 12, 4, 4096
    counts = np.zeros(V)
    g = np.random.Generator(np.random.PCG64(99))
    row = g.standard_normal(V).astype(np.float32) * 1.2
    q = (row + 1.0 * g.standard_normal(V)).astype(np.float32)
    pq = np.exp(q - q.max()) / np.exp(q - q.max()).sum()
    for rep in range(3):
        c = dict(target=torch.from_numpy(np.tile(row, (B, n, 1))), parents=np.tile(np.array([-1, 0, 0, 0], np.int32), (B, 1)),
                 draft=torch.from_numpy(np.tile(q, (B, n, 1))) if drawn else None, n_nodes=None, temperature=None,
                 uniforms=g.random((B, n), dtype=np.float32),
                 noise=g.standard_exponential((B, V)).astype(np.float32) + np.float32(1e-12))
        c["tokens"] = g.choice(V, size=(B, n), p=pq).astype(np.int32) if drawn else \
            np.tile(np.array([0, 3, 7, 5], np.int32), (B, 1))
        counts += np.bincount(_run(c)[0][:, 0], minlength=V)
    p = np.exp(row.astype(np.float64) - row.max())
    p /= p.sum()
    want = p * 3 * B
    assert ((counts - want) ** 2 / want).sum() < 37.4


def test_workspace_reused_and_graph_replay():
    c = _inputs(30, 7, 16, 20001, "bf16", True)
    want = _run(c)
    ws = vq.Workspace(vq.tree_verify_workspace_bytes(7, 16, 20001))
    ws.tensor.fill_(0xFF)
    for x, y in zip(_run(c, workspace=ws), want):
        assert np.array_equal(x, y)
    dev = {k: _dev(x) for k, x in c.items()}
    outs = [torch.empty(7, 16, dtype=torch.int32, device="cuda") for _ in range(2)] + \
        [torch.empty(7, dtype=torch.int32, device="cuda")]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        vq.tree_verify(dev["target"], dev["draft"], dev["tokens"], dev["uniforms"], dev["noise"],
                       parents=dev["parents"], temperature=dev["temperature"], tokens_out=outs[0], path_out=outs[1],
                       count_out=outs[2], workspace=ws)
    for _ in range(4):
        for o in outs:
            o.fill_(-9)
        ws.tensor.fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert np.array_equal(x.cpu().numpy(), y)
