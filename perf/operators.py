"""Cases of the operators around the verify GEMMs of a speculative-decoding
step: attention of drafted tokens over a paged cache, acceptance of a draft
tree from given random numbers, and writing keys and values into the cache.

`run` computes a case in plain torch operations (own = False) or with the
library's entry points (own = True) on the state that `prepare` makes.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32  # tokens per transposed block of the value cache


# ------------------------------------------------------------------ the cases

def listed():
    """Attention: 64 query heads of 128 make the 8192-wide projections of the
    weight stream; 16 nodes are a full draft block of the verify GEMMs.
    Acceptance: 151,936 is the vocabulary of the greedy measurement.  Append:
    16 layers, keys and values of 8 heads of 128."""
    return [
        # one user's short chat, a chain of 8 drafted tokens: latency counts
        dict(name="attn chain 1x8 ctx 509", op="attn", batch=1, n=8, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", ctx_lo=509, ctx=509, tree="chain", ragged=False, fused=True),
        # plain decoding of a served batch: single tokens, ragged contexts
        dict(name="attn decode 32x1 ctx 4k", op="attn", batch=32, n=1, heads=32, kv_heads=8, dim=64, page=32,
             dtype="f16", ctx_lo=1, ctx=4096, tree="chain", ragged=False, fused=True),
        # a served batch verifying 16-node trees, ragged contexts
        dict(name="attn tree 8x16 ctx 16k", op="attn", batch=8, n=16, heads=64, kv_heads=8, dim=128, page=64,
             dtype="bf16", ctx_lo=1024, ctx=16384, tree="tree", ragged=True, fused=True),
        # one user with a long document
        dict(name="attn tree 1x16 ctx 128k", op="attn", batch=1, n=16, heads=64, kv_heads=8, dim=128, page=128,
             dtype="bf16", ctx_lo=131071, ctx=131071, tree="tree", ragged=False, fused=True),
        # wide trees (odd size), wide heads: many query rows for each cached token
        dict(name="attn tree 4x61 ctx 8k", op="attn", batch=4, n=61, heads=32, kv_heads=4, dim=256, page=64,
             dtype="f16", ctx_lo=777, ctx=8191, tree="tree", ragged=True, fused=False),
        # one user, a chain of 15 tokens drawn from the drafter's distributions
        dict(name="verify chain 1x16 V 152k", op="verify", batch=1, n=16, vocab=151936, dtype="bf16", tree="chain",
             branch=1, ragged=False, sampled=True, greedy_every=0),
        # a few users, wide trees of the drafter's best tokens (no distributions), odd vocabulary
        dict(name="verify tree 4x61 V 32001", op="verify", batch=4, n=61, vocab=32001, dtype="f32", tree="tree",
             branch=6, ragged=True, sampled=False, greedy_every=0),
        # a served batch of sampled trees, every fourth user decoding greedily
        dict(name="verify tree 32x16 V 152k", op="verify", batch=32, n=16, vocab=151936, dtype="bf16", tree="tree",
             branch=3, ragged=True, sampled=True, greedy_every=4),
        # commit of one user's accepted path in all layers
        dict(name="append path 1x16 16 layers", op="append", layers=16, batch=1, n=16, kv_heads=8, dim=128, page=64,
             dtype="bf16", ctx_lo=4093, ctx=4093, path=True, fused=False),
        # commit of a served batch's accepted paths in all layers
        dict(name="append path 32x16 16 layers", op="append", layers=16, batch=32, n=16, kv_heads=8, dim=128, page=64,
             dtype="bf16", ctx_lo=100, ctx=2048, path=True, fused=False),
        # two prompts' keys and values into one layer's pages, straight from the fused projection
        dict(name="append prompt 2x8190", op="append", layers=1, batch=2, n=8190, kv_heads=8, dim=128, page=64,
             dtype="f16", ctx_lo=0, ctx=37, path=False, fused=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "verify", "append"])
    if op == "attn":
        tree = rng.choice(["chain", "tree"])
        c = dict(op=op, batch=_log_int(rng, 1, 32), n=_log_int(rng, 1, 64), kv_heads=rng.choice([1, 2, 4, 8]), heads=0,
                 dim=rng.choice([64, 128, 256]), page=rng.choice([32, 64, 128, 256]),
                 dtype=rng.choice(["bf16", "f16"]), ctx_lo=0, ctx=_log_int(rng, 1, 131072), tree=tree,
                 ragged=rng.random() < 0.5, fused=rng.random() < 0.5)
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8])
        # no more cached elements and no more scores than the largest listed case
        most = min((131071 * 8 * 128) // (c["batch"] * c["kv_heads"] * c["dim"]),
                   (131071 * 64 * 16) // (c["batch"] * c["heads"] * c["n"]))
        c["ctx"] = min(c["ctx"], most)
        c["ctx_lo"] = rng.randint(0, c["ctx"])
        return c
    if op == "verify":
        tree = rng.choice(["chain", "tree"])
        c = dict(op=op, batch=_log_int(rng, 1, 32), n=_log_int(rng, 2, 64), vocab=_log_int(rng, 1000, 151936),
                 dtype=rng.choice(["bf16", "f16", "f32"]), tree=tree, branch=1 if tree == "chain" else rng.randint(2, 6),
                 ragged=rng.random() < 0.5, sampled=rng.random() < 0.6, greedy_every=rng.choice([0, 0, 2, 5]))
        most = (32 * 16 * 151936) // (c["batch"] * c["vocab"] * (2 if c["dtype"] == "f32" else 1))
        c["n"] = max(2, min(c["n"], most))
        return c
    path = rng.random() < 0.6
    c = dict(op=op, layers=_log_int(rng, 1, 16) if path else 1, batch=_log_int(rng, 1, 32),
             n=_log_int(rng, 1, 64) if path else _log_int(rng, 1, 8190), kv_heads=rng.choice([1, 2, 4, 8]),
             dim=rng.choice([64, 128, 256]), page=rng.choice([32, 64, 128, 256]), dtype=rng.choice(["bf16", "f16"]),
             ctx_lo=0, ctx=_log_int(rng, 1, 2048), path=path, fused=rng.random() < 0.5)
    most = (2 * 8190 * 8 * 128) // (c["layers"] * c["batch"] * c["kv_heads"] * c["dim"])
    c["n"] = max(1, min(c["n"], most))
    c["ctx_lo"] = rng.randint(0, c["ctx"])
    return c


# ------------------------------------------------------------------ inputs

def _spread(lo, hi, count, at_most):
    """`count` whole numbers spread over lo .. hi, the first of them hi."""
    return [min(at_most, hi - int((hi - lo) * ((0.6180339887 * b) % 1.0))) for b in range(count)]


def _ctx_lens(case):
    return _spread(case["ctx_lo"], case["ctx"], case["batch"], case["ctx"])


def _node_counts(case):
    n = case["n"]
    return _spread(max(1, n // 2), n, case["batch"], n) if case.get("ragged") else [n] * case["batch"]


def _path_counts(case):
    """Accepted rows of each sequence: up to half of the tree."""
    return _spread(1, max(1, case["n"] // 2), case["batch"], case["n"])


def _trees(case, g):
    """Random trees int64 [B][n]: each node hangs on one of the last nodes
    before it that has room for a child."""
    parents = np.zeros((case["batch"], case["n"]), dtype=np.int64)
    for b in range(case["batch"]):
        free = [case.get("branch", 4)]
        parents[b, 0] = -1
        for i in range(1, case["n"]):
            room = [v for v in range(i) if free[v] > 0][-8:]
            v = room[g.randint(len(room))]
            free[v] -= 1
            free.append(case.get("branch", 4))
            parents[b, i] = v
    return parents


def _ancestors(parents):
    """bool [B][n][n]: whether j is i or one of its ancestors."""
    B, n = parents.shape
    a = np.zeros((B, n, n), dtype=bool)
    for b in range(B):
        for i in range(n):
            if i > 0:
                a[b, i] = a[b, parents[b, i]]
            a[b, i, i] = True
    return a


def _chain(case):
    return np.tile(np.arange(case["n"]) - 1, (case["batch"], 1))


def _pages(case, lens, g, dev):
    """A page table for `lens` tokens of each sequence over a shuffled pool; -1 past a sequence's pages."""
    page = case["page"]
    need = [max(1, -(-x // page)) for x in lens]
    pool = g.permutation(sum(need) + 3)
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = pool[at:at + k]
        at += k
    return torch.from_numpy(table).to(dev), len(pool)


def _rows(shape_bn, widths, fused, dtype, gen, dev):
    """Projection outputs of widths[i] for each row: views of one fused matrix, or matrices of their own."""
    if fused:
        m = torch.randn(*shape_bn, sum(widths), generator=gen, device=dev, dtype=torch.float32).to(dtype)
        return list(torch.split(m, widths, dim=-1))
    return [torch.randn(*shape_bn, w, generator=gen, device=dev, dtype=torch.float32).to(dtype) for w in widths]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    g = np.random.RandomState(int(seed) % (1 << 31))
    st = dict(op=case["op"], case=case)
    if case["op"] == "verify":
        st.update(_prepare_verify(case, gen, g, dev))
        return st
    dt = DTYPES[case["dtype"]]
    B, n, H, D = case["batch"], case["n"], case["kv_heads"], case["dim"]
    lens = np.array(_ctx_lens(case), dtype=np.int32)[g.permutation(B)]
    st["page_table"], pages = _pages(case, [int(x) + n for x in lens], g, dev)
    st["ctx_len"] = torch.from_numpy(lens).to(dev)
    lead = (case["layers"],) if case["op"] == "append" else ()
    # pages hold earlier tokens and, past them, what other sequences left there
    st["k_cache"] = torch.randn(*lead, pages, H, case["page"], D, generator=gen, device=dev, dtype=dt)
    st["v_cache"] = torch.randn(*lead, pages, H, case["page"] // BLOCK, D, BLOCK, generator=gen, device=dev, dtype=dt)
    if case["op"] == "append":
        k, v = _rows((*lead, B, n), [H * D, H * D], case["fused"], dt, gen, dev)
        st["k"], st["v"] = k.unflatten(-1, (H, D)), v.unflatten(-1, (H, D))
        st["path"] = st["count"] = None
        if case["path"]:
            counts = np.array(_path_counts(case), dtype=np.int32)[g.permutation(B)]
            path = np.full((B, n), -1, dtype=np.int32)
            for b in range(B):
                path[b, :counts[b]] = np.concatenate([[0], 1 + np.sort(g.permutation(n - 1)[:counts[b] - 1])])
            st["path"], st["count"] = torch.from_numpy(path).to(dev), torch.from_numpy(counts).to(dev)
        return st
    q, k, v = _rows((B, n), [case["heads"] * D, H * D, H * D], case["fused"], dt, gen, dev)
    st["q"] = q.unflatten(-1, (case["heads"], D))
    st["k"], st["v"] = k.unflatten(-1, (H, D)), v.unflatten(-1, (H, D))
    st["n_nodes"] = torch.tensor(_node_counts(case), dtype=torch.int32)[torch.from_numpy(g.permutation(B))].to(dev) \
        if case["ragged"] else None
    st["tree_mask"] = None
    if case["tree"] == "tree":
        bits = _ancestors(_trees(case, g)).astype(np.uint64) << np.arange(n, dtype=np.uint64)
        st["tree_mask"] = torch.from_numpy(bits.sum(-1, dtype=np.uint64).view(np.int64)).to(dev)
    return st


def _prepare_verify(case, gen, g, dev):
    """Target rows with a heavy tail (the probability of the token of rank r
    falls as r^-1.3), drafter rows near them; children drawn from the
    drafter's row of their parent, or its best tokens."""
    dt = DTYPES[case["dtype"]]
    B, n, V = case["batch"], case["n"], case["vocab"]
    parents = _trees(case, g) if case["tree"] == "tree" else _chain(case)
    target = torch.empty(B, n, V, device=dev, dtype=dt)
    draft = torch.empty(B, n, V, device=dev, dtype=dt) if case["sampled"] else None
    tokens = torch.zeros(B, n, dtype=torch.int32, device=dev)
    temps = 0.6 + 0.6 * g.random_sample(B)
    rank = np.zeros((B, n), dtype=np.int64)  # which child of its parent a node is
    for b in range(B):
        seen = {}
        for i in range(1, n):
            rank[b, i] = seen.get(parents[b, i], 0)
            seen[parents[b, i]] = rank[b, i] + 1
    up = torch.from_numpy(parents).clamp(min=0).to(dev)
    for b in range(B):
        t = -1.3 * torch.log(torch.rand(n, V, generator=gen, device=dev).clamp(min=1e-9))
        d = t + 0.7 * torch.randn(n, V, generator=gen, device=dev)
        target[b] = t.to(dt)
        if draft is not None:
            draft[b] = d.to(dt)
            e = torch.empty(n, V, device=dev).exponential_(generator=gen)
            x = (draft[b].float() / temps[b])[up[b]] - torch.log(e)
            tokens[b] = x.argmax(-1).to(torch.int32)
        else:
            best = d.topk(min(V, max(1, case["branch"])), dim=-1).indices[up[b]]
            at = torch.from_numpy(rank[b]).to(dev)
            tokens[b] = best.gather(1, at[:, None])[:, 0].to(torch.int32)
    if case["greedy_every"]:
        temps[::case["greedy_every"]] = 0.0
    return dict(
        target=target, draft=draft, tokens=tokens,
        parents=torch.from_numpy(parents.astype(np.int32)).to(dev) if case["tree"] == "tree" else None,
        n_nodes=torch.tensor(_node_counts(case), dtype=torch.int32, device=dev) if case["ragged"] else None,
        temperature=torch.from_numpy(temps.astype(np.float32)).to(dev),
        uniforms=torch.rand(B, n, generator=gen, device=dev),
        noise=torch.empty(B, V, device=dev).exponential_(generator=gen))


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    return {"attn": _plain_attn, "verify": _plain_verify, "append": _plain_append}[st["op"]](st)


def _run_own(st):
    import block_quantized_gemm_amd as vq
    if st["op"] == "attn":
        return vq.tree_attention(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"],
                                 st["ctx_len"], tree_mask=st["tree_mask"], n_nodes=st["n_nodes"])
    if st["op"] == "verify":
        return vq.tree_verify(st["target"], st["draft"], st["tokens"], st["uniforms"], st["noise"],
                              parents=st["parents"], n_nodes=st["n_nodes"], temperature=st["temperature"])
    new_len = vq.kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["page_table"], st["ctx_len"],
                           path=st["path"], count=st["count"])
    return st["k_cache"], st["v_cache"], new_len


def _plain_attn(st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    B, n, Hq, D = q.shape
    H = k.shape[2]
    table = st["page_table"].long().clamp(min=0)
    kc = st["k_cache"][table].float()                            # [B][W][H][page][D]
    vc = st["v_cache"][table].float().transpose(-1, -2)          # [B][W][H][page/32][32][D]
    T = kc.shape[1] * kc.shape[3]
    kc = kc.transpose(1, 2).reshape(B, H, T, D)
    vc = vc.permute(0, 2, 1, 3, 4, 5).reshape(B, H, T, D)
    kt = torch.cat([kc, k.transpose(1, 2)], 2).transpose(-1, -2).contiguous()
    vt = torch.cat([vc, v.transpose(1, 2)], 2)
    node = torch.arange(n, device=q.device)
    bits = (st["tree_mask"][:, :, None] >> node) & 1 if st["tree_mask"] is not None else \
        (node[None, :] <= node[:, None]).long().expand(B, n, n)
    live = (node < (st["n_nodes"][:, None] if st["n_nodes"] is not None else n)).expand(B, n)
    tree = (bits == 1) & live[:, None, :]
    past = torch.arange(T, device=q.device)[None, None, :] < st["ctx_len"][:, None, None]
    seen = torch.cat([past.expand(B, n, T), tree], 2) & live[:, :, None]
    qs = q.view(B, n, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * (Hq // H), D)
    s = torch.matmul(qs, kt) * (1.0 / math.sqrt(D))
    s = s.view(B, H, n, Hq // H, T + n).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, -1, T + n), vt).view(B, H, n, Hq // H, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D).to(st["q"].dtype)


def _softmax(x, temperature):
    x = x.float() / torch.where(temperature > 0, temperature, torch.ones_like(temperature))[:, None, None]
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_verify(st):
    case, tokens = st["case"], st["tokens"].long()
    B, n, V = st["target"].shape
    dev = tokens.device
    node = torch.arange(n, device=dev)
    up = st["parents"].long() if st["parents"] is not None else (node - 1).expand(B, n)
    live = (node < (st["n_nodes"][:, None] if st["n_nodes"] is not None else n)).expand(B, n)
    greedy = st["temperature"] == 0
    p = _softmax(st["target"], st["temperature"])
    q = _softmax(st["draft"], st["temperature"]) if st["draft"] is not None else None
    best = st["target"].argmax(-1)
    # is_child[b][v][c]; order[b][v][c] = how many children v has before c
    is_child = (up[:, None, :] == node[None, :, None]) & live[:, None, :] & (node[None, None, :] > 0)
    order = is_child.long().cumsum(-1) - 1
    chosen = torch.full((B, n), -1, dtype=torch.long, device=dev)
    S, s = torch.zeros(B, n, device=dev), torch.ones(B, n, device=dev)
    r = p
    for j in range(case["branch"]):
        at = is_child & (order == j)
        tried = at.any(-1) & (chosen < 0)
        c = at.long().argmax(-1)
        x = tokens.gather(1, c)
        u = st["uniforms"].gather(1, c)
        rx = r.gather(2, x[:, :, None])[:, :, 0]
        qx = q.gather(2, x[:, :, None])[:, :, 0] if q is not None else 1.0
        ok = torch.where(greedy[:, None], x == best, u * qx * s < rx) & tried
        chosen = torch.where(ok, c, chosen)
        no = tried & ~ok
        S = torch.where(no, S + s, S)
        if q is not None:
            r = torch.clamp(p - S[:, :, None] * q, min=0)
            s = torch.where(no & (S > 0), r.sum(-1), s)
        else:
            r = r.scatter(2, x[:, :, None], torch.where(no, torch.zeros_like(rx), rx)[:, :, None])
            s = torch.where(no, s - rx, s)
    # a node is reached when it and its ancestors were chosen by their parents
    accepted = (chosen.gather(1, up.clamp(min=0)) == node) | (node == 0)
    hop = torch.nn.functional.one_hot(up.clamp(min=0), n).float()  # parent of each node; the root is its own
    reach = accepted.float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = reach * torch.matmul(hop, reach[:, :, None])[:, :, 0]
        hop = torch.matmul(hop, hop)
    reached = (reach > 0) & live
    count = reached.sum(-1)
    path = torch.where(reached, node, n).sort(-1).values
    last = path.gather(1, (count - 1)[:, None])[:, 0]
    row = torch.arange(B, device=dev)
    rest = r[row, last]
    rest = torch.where((rest > 0).any(-1, keepdim=True), rest, p[row, last])
    final = torch.where(greedy, best[row, last], (rest / st["noise"]).argmax(-1))
    after = torch.cat([path[:, 1:], torch.full((B, 1), n, device=dev)], 1)
    out = tokens.gather(1, after.clamp(max=n - 1))
    out = torch.where(node == (count - 1)[:, None], final[:, None], out)
    done = node >= count[:, None]
    return (out.masked_fill(done, -1).int(), path.masked_fill(done, -1).int(), count.int())


def _plain_append(st):
    k, v = st["k"], st["v"]
    B, n = k.shape[1:3]
    page = st["case"]["page"]
    dev = k.device
    i = torch.arange(n, device=dev)
    count = st["count"].long() if st["count"] is not None else torch.full((B,), n, device=dev)
    src = st["path"].long() if st["path"] is not None else i.expand(B, n)
    b, at = torch.nonzero(i < count[:, None], as_tuple=True)
    row = src[b, at]
    pos = st["ctx_len"].long()[b] + at
    pg = st["page_table"].long()[b, pos // page]
    off = pos % page
    st["k_cache"][:, pg, :, off] = k[:, b, row].transpose(0, 1)
    st["v_cache"][:, pg, :, off // BLOCK, :, off % BLOCK] = v[:, b, row].transpose(0, 1)
    return st["k_cache"], st["v_cache"], (st["ctx_len"].long() + count).int()


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "attn":
        e = 2
        B, n, Hq, H, D = case["batch"], case["n"], case["heads"], case["kv_heads"], case["dim"]
        lens, nodes = _ctx_lens(case), _node_counts(case)
        rows = sum(nodes) * (2 * Hq + 2 * H) * D * e  # queries and outputs, drafted keys and values
        # every node sees the whole context and itself at least (a permutation pairs them, so by their means)
        pairs = sum(nodes) * (sum(lens) / B + 1)
        return {"bytes": sum(lens) * H * D * 2 * e + rows, "flops": 4 * D * Hq * pairs}
    if case["op"] == "verify":
        e = 4 if case["dtype"] == "f32" else 2
        rows = sum(_node_counts(case)) * case["vocab"]
        # the drafter's rows of leaves are not needed: at least one node in `branch` has children
        inner = rows / case["branch"] if case["sampled"] else 0
        return {"bytes": (rows + inner) * e + case["batch"] * case["vocab"] * 4, "flops": 4 * (rows + inner)}
    rows = sum(_path_counts(case)) if case["path"] else case["batch"] * case["n"]
    return {"bytes": 2 * 2 * 2 * rows * case["layers"] * case["kv_heads"] * case["dim"], "flops": 0}


# ------------------------------------------------------------------ from the definition, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, st)
    if case["op"] == "verify":
        return _exact_verify(case, st)
    return None  # copies


def _exact_attn(case, st):
    B, n, Hq, H, D = case["batch"], case["n"], case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64, device="cuda")
    masks = st["tree_mask"].cpu().numpy().view(np.uint64) if st["tree_mask"] is not None else None
    nodes = st["n_nodes"].tolist() if st["n_nodes"] is not None else [n] * B
    for b in range(B):
        ctx = int(st["ctx_len"][b])
        ids = [int(x) for x in st["page_table"][b, :-(-ctx // case["page"])]]
        for h in range(H):
            keys = [st["k_cache"][ids, h].reshape(-1, D)[:ctx], st["k"][b, :nodes[b], h]]
            vals = [st["v_cache"][ids, h].permute(0, 1, 3, 2).reshape(-1, D)[:ctx], st["v"][b, :nodes[b], h]]
            keys, vals = (torch.cat([x.double() for x in xs]) for xs in (keys, vals))
            for i in range(nodes[b]):
                bits = int(masks[b, i]) if masks is not None else (1 << (i + 1)) - 1
                sel = torch.tensor([ctx + j for j in range(nodes[b]) if bits >> j & 1], dtype=torch.long, device=out.device)
                kk, vv = (torch.cat([x[:ctx], x[sel]]) for x in (keys, vals))
                if kk.shape[0] == 0:
                    continue
                hq = slice(h * (Hq // H), (h + 1) * (Hq // H))
                w = torch.softmax(kk @ st["q"][b, i, hq].double().t() / math.sqrt(D), 0)
                out[b, i, hq] = w.t() @ vv
    return out


def _exact_verify(case, st):
    B, n = case["batch"], case["n"]
    nodes = st["n_nodes"].tolist() if st["n_nodes"] is not None else [n] * B
    tokens, u = st["tokens"].tolist(), st["uniforms"].double().tolist()
    parents = st["parents"].tolist() if st["parents"] is not None else _chain(case).tolist()
    out, paths = np.full((B, n), -1, dtype=np.int32), np.full((B, n), -1, dtype=np.int32)
    counts = np.zeros(B, dtype=np.int32)
    for b in range(B):
        temp = float(st["temperature"][b])
        path, final = [0], None
        while final is None:
            v = path[-1]
            logits = st["target"][b, v].double()
            kids = [c for c in range(1, nodes[b]) if parents[b][c] == v]
            if temp == 0:
                top = int(logits.argmax())
                took = next((c for c in kids if tokens[b][c] == top), None)
                final = top if took is None else None
            else:
                left = p = torch.softmax(logits / temp, 0)
                took = None
                for c in kids:
                    x = tokens[b][c]
                    if st["draft"] is not None:
                        q = torch.softmax(st["draft"][b, v].double() / temp, 0)
                    else:
                        q = torch.zeros_like(p)
                        q[x] = 1.0
                    if u[b][c] * float(q[x]) < float(left[x]):
                        took = c
                        break
                    left = torch.clamp(left - q, min=0)
                    left = left / left.sum()
                if took is None:
                    final = int((left / st["noise"][b].double()).argmax())
            if took is not None:
                path.append(took)
        counts[b] = len(path)
        paths[b, :len(path)] = path
        out[b, :len(path)] = [tokens[b][c] for c in path[1:]] + [final]
    return out, paths, counts
