"""Tree attention on the GPU against the definition at 64 bits."""
import numpy as np
import pytest
import torch

import block_quantized_gemm_amd as vq
import tree_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Case:
    """Inputs of one call: random rows, a shuffled page pool, stale values past every sequence's tokens."""

    def __init__(self, seed, dtype, n, Hq, H, D, page, lens, nodes=None, mask="tree", fused=False, spare=2,
                 amplitude=1.0):
        g = np.random.Generator(np.random.PCG64(seed))
        gen = torch.Generator().manual_seed(seed)
        self.dtype, self.scale = dtype, D ** -0.5
        dt, B = DT[dtype], len(lens)

        def rand(*shape):
            return torch.randn(*shape, generator=gen).to(dt)

        need = [max(1, -(-x // page)) for x in lens]
        W = max(need) + 1
        pool = g.permutation(sum(need) + spare)
        table = np.full((B, W), -1, np.int32)
        at = 0
        for b, c in enumerate(need):
            table[b, :c] = pool[at:at + c]
            at += c
            table[b, c:] = [-1, 1 << 20, -(1 << 31)][b % 3]  # never read
        P = len(pool)
        self.k_cache, self.v_cache = rand(P, H, page, D), rand(P, H, page // 32, D, 32)
        if fused:
            m = rand(B, n, (Hq + 2 * H) * D + 8)[..., :(Hq + 2 * H) * D]  # a row stride wider than the row
            q, k, v = torch.split(m, [Hq * D, H * D, H * D], dim=-1)
        else:
            q, k, v = rand(B, n, Hq * D), rand(B, n, H * D), rand(B, n, H * D)
        self.q, self.k, self.v = q.unflatten(-1, (Hq, D)) * 1, k.unflatten(-1, (H, D)), v.unflatten(-1, (H, D))
        if fused:
            self.q = q.unflatten(-1, (Hq, D))
        elif amplitude != 1.0:
            self.q = (self.q * amplitude).to(dt)
        self.table, self.lens = table, np.array(lens, np.int32)
        self.nodes = None if nodes is None else np.array(nodes, np.int32)
        if mask == "tree":
            self.masks = R.ancestor_masks(R.random_trees(B, n, g))
        elif mask == "random":
            self.masks = g.integers(0, 1 << 63, size=(B, n), dtype=np.uint64) * np.uint64(2) + np.uint64(1)
            self.masks[:, ::3] = 0  # rows that see no node
        else:
            self.masks = None

    def poison(self):
        """Infinities and NaN wherever nothing may look: the cache past every
        sequence's tokens, and the nodes past n_nodes."""
        page = self.k_cache.shape[2]
        used = np.zeros((self.k_cache.shape[0], page), bool)
        for b, x in enumerate(self.lens):
            for t in range(int(x)):
                used[self.table[b, t // page], t % page] = True
        bad = torch.from_numpy(~used)
        self.k_cache[bad[:, None, :].expand(-1, self.k_cache.shape[1], -1)] = float("nan")
        vb = bad.view(bad.shape[0], 1, page // 32, 1, 32).expand(self.v_cache.shape)
        self.v_cache[vb] = float("inf")
        if self.nodes is not None:
            for b, x in enumerate(self.nodes):
                self.k[b, int(x):] = float("-inf")
                self.v[b, int(x):] = float("nan")
                self.q[b, int(x):] = float("nan")
        return self

    def run(self, stream=None, workspace="auto"):
        dev = [None if t is None else t.cuda() if isinstance(t, torch.Tensor) else torch.from_numpy(t).cuda()
               for t in (self.k_cache, self.v_cache, self.table, self.lens, self.nodes,
                         None if self.masks is None else self.masks.view(np.int64))]
        kc, vc, table, lens, nodes, masks = dev

        def rows(t):  # keep the row stride of a fused projection
            if t.is_contiguous():
                return t.cuda()
            return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)
        args = rows(self.q), rows(self.k), rows(self.v), kc, vc, table, lens
        torch.cuda.synchronize()
        out = vq.tree_attention(*args, tree_mask=masks, n_nodes=nodes, scale=self.scale, stream=stream,
                                workspace=workspace)
        torch.cuda.synchronize()
        return out.cpu()

    def ref(self):
        clean = [np.nan_to_num(_f64(t), nan=0.0, posinf=0.0, neginf=0.0)
                 for t in (self.q, self.k, self.v, self.k_cache, self.v_cache)]
        return R.attention(*clean, self.table, self.lens, self.masks, self.nodes, self.scale, self.dtype)

    def check(self, out=None):
        y = _f64(self.run() if out is None else out)
        ref, bound = self.ref()
        assert np.isfinite(y).all()
        worst = np.max(np.abs(y - ref) / np.maximum(bound, 1e-300))
        assert (np.abs(y - ref) <= bound).all(), "error %.2f of the bound" % worst
        return y


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 32), (128, 64), (256, 128), (128, 256)])
@pytest.mark.parametrize("n,Hq,H,lens,mask", [
    (1, 1, 1, [1], None), (1, 8, 2, [0, 31, 32, 33, 700], None), (8, 6, 2, [257, 0, 64], None),
    (16, 8, 1, [100, 1025], "tree"), (5, 5, 5, [63, 95], "tree"), (33, 4, 2, [40, 129], "random"),
    (64, 3, 1, [0, 300], "tree")])
def test_shapes(dtype, D, page, n, Hq, H, lens, mask):
    Case(7 + n + D + page, dtype, n, Hq, H, D, page, lens, mask=mask).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,lens,nodes", [(4, [33, 0, 70], [4, 1, 0]), (40, [5, 64, 0], [33, 40, 17]),
                                          (64, [1, 2], [64, 63])])
def test_ragged_nodes_and_poison(dtype, n, lens, nodes):
    """n_nodes below n; NaN and infinities everywhere a row may not look."""
    for mask in (None, "tree", "random"):
        c = Case(50 + n, dtype, n, 4, 2, 128, 64, lens, nodes=nodes, mask=mask).poison()
        y = c.check()
        for b, x in enumerate(nodes):
            assert (y[b, x:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [6, 40])
def test_unseen_nodes_may_hold_anything(dtype, n):
    """A node that only some rows see may hold infinities and NaN: the other
    rows' outputs are those without it."""
    for what in (float("inf"), float("-inf"), float("nan")):
        c = Case(77, dtype, n, 4, 1, 64, 32, [37, 0], mask="tree")
        bad = n - 2
        sees = (c.masks >> np.uint64(bad)) & np.uint64(1) == 1
        clean = Case(77, dtype, n, 4, 1, 64, 32, [37, 0], mask="tree").run()
        c.k[:, bad], c.v[:, bad] = what, what
        out = c.run()
        keep = torch.from_numpy(~sees)
        assert torch.equal(out[keep], clean[keep])
        assert not torch.isfinite(out[torch.from_numpy(sees)]).all(-1).any()
    c = Case(78, dtype, n, 4, 1, 64, 32, [37, 0], mask="tree")
    c.v[:, n - 2, :, 5] = float("inf")  # one channel: only that channel of the rows that see it
    sees = torch.from_numpy((c.masks >> np.uint64(n - 2)) & np.uint64(1) == 1)
    clean = Case(78, dtype, n, 4, 1, 64, 32, [37, 0], mask="tree").run()
    out = c.run()
    assert (out[sees][..., 5] == float("inf")).all()
    other = torch.arange(64) != 5
    assert torch.equal(out[..., other], clean[..., other]) and torch.equal(out[~sees], clean[~sees])


def test_rows_that_see_nothing_are_zero():
    c = Case(80, "bf16", 7, 4, 2, 128, 64, [0, 0], mask="random")
    c.masks[0] = 0
    y = c.check()
    assert (y[0] == 0).all() and (y[1, ::3] == 0).all() and (np.abs(y[1, 1]).sum() > 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_scores(dtype):
    """Scores of hundreds, both signs: the running maximum moves often, most probabilities vanish."""
    Case(81, dtype, 9, 4, 2, 128, 64, [300, 77], mask="tree", amplitude=60.0).check()


def test_growing_scores():
    """Scores that keep growing with the position, past any fixed head room."""
    c = Case(82, "bf16", 3, 2, 1, 64, 32, [640], mask=None)
    page = 32
    for t in range(640):
        c.k_cache[int(c.table[0, t // page]), 0, t % page] = 0
        c.k_cache[int(c.table[0, t // page]), 0, t % page, 0] = float(t)
    c.q[...] = 0
    c.q[..., 0] = 4.0
    c.check()
    c.q[..., 0] = -4.0
    c.check()


def test_fused_rows():
    for n, Hq, H in ((1, 4, 1), (16, 8, 2)):
        c = Case(83, "bf16", n, Hq, H, 128, 64, [130, 9], fused=True)
        assert not c.q.is_contiguous() or n * len(c.lens) == 1
        c.check()


@pytest.mark.parametrize("D,Hq,H,n,L", [(128, 8, 1, 16, 4500), (64, 2, 1, 1, 9001), (256, 4, 1, 20, 2600)])
def test_long_contexts(D, Hq, H, n, L):
    """Contexts that are cut between workgroups and joined again, beside a short one."""
    Case(84, "bf16", n, Hq, H, D, 64, [L, 3, L - 129], mask="tree").check()


def test_many_sequences():
    lens = [int(x) for x in np.random.Generator(np.random.PCG64(5)).integers(0, 120, size=300)]
    Case(85, "f16", 2, 2, 1, 64, 32, lens, mask=None).check()


def test_same_bits_any_workspace_any_stream():
    c = Case(86, "bf16", 12, 8, 2, 128, 64, [2000, 15, 700], mask="tree")
    first = c.run()
    c.check(first)
    ws = vq.Workspace(vq.tree_attention_workspace_bytes(3, 12, 8, 2, 128))
    ws.tensor.fill_(0xFF)
    assert torch.equal(c.run(workspace=ws), first)
    assert torch.equal(c.run(workspace=ws), first)
    assert torch.equal(c.run(stream=torch.cuda.Stream()), first)


def test_pages_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, the sequence's pages at its end."""
    H, page, D, L = 8, 256, 128, 600
    P = (1 << 31) // (H * page * D) + 8
    c = Case(87, "bf16", 4, 16, 8, D, page, [L], mask="tree", spare=0)
    kc = torch.empty(P, H, page, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty(P, H, page // 32, D, 32, dtype=torch.bfloat16, device="cuda")
    at = [P - 1, P - 5, P - 3]
    table = np.full((1, 4), -1, np.int32)
    for j in range(3):
        kc[at[j]] = c.k_cache[int(c.table[0, j])].cuda()
        vc[at[j]] = c.v_cache[int(c.table[0, j])].cuda()
        table[0, j] = at[j]
    out = vq.tree_attention(c.q.cuda(), c.k.cuda(), c.v.cuda(), kc, vc, torch.from_numpy(table).cuda(),
                            torch.from_numpy(c.lens).cuda(),
                            tree_mask=torch.from_numpy(c.masks.view(np.int64)).cuda(), scale=c.scale)
    c.check(out)


def test_length_past_the_table_is_cut():
    c = Case(88, "bf16", 3, 4, 2, 64, 32, [64], mask=None)
    c.table = np.ascontiguousarray(c.table[:, :2])
    want = c.run()
    c.lens[0] = 70
    assert torch.equal(c.run(), want)
    c.check()
    c.lens[0] = -5
    c.check()


def test_bad_page_reads_as_zeros():
    c = Case(89, "bf16", 3, 4, 2, 64, 32, [100], mask=None)
    c.table[0, 1] = 1 << 24
    c.check()


def test_graph_replay():
    c = Case(90, "bf16", 8, 8, 2, 128, 64, [900, 40], mask="tree")
    want = c.run()
    dev = [t.cuda() for t in (c.q, c.k, c.v, c.k_cache, c.v_cache, torch.from_numpy(c.table), torch.from_numpy(c.lens))]
    masks = torch.from_numpy(c.masks.view(np.int64)).cuda()
    ws = vq.Workspace(vq.tree_attention_workspace_bytes(2, 8, 8, 2, 128))
    out = torch.empty_like(dev[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        vq.tree_attention(*dev, tree_mask=masks, scale=c.scale, out=out, workspace=ws)
    for _ in range(4):
        out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)
        ws.tensor.fill_(0x5A)
