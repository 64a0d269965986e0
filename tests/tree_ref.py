"""The speculative-step operators from their definitions, in numpy at 64 bits.

Plain loops over sequences, heads and nodes; nothing here is shared with the
library or with the benchmark's plain forms."""
from __future__ import annotations

import math

import numpy as np

# Half of the relative spacing of the output types: the largest relative error
# of one rounding.
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def cached_rows(k_cache, v_cache, table_row, h, length, page):
    """Keys and values [length][D] of one sequence and head, float64."""
    D = k_cache.shape[-1]
    k, v = np.zeros((length, D)), np.zeros((length, D))
    for t in range(length):
        pg = int(table_row[t // page])
        if 0 <= pg < k_cache.shape[0]:
            off = t % page
            k[t] = k_cache[pg, h, off]
            v[t] = v_cache[pg, h, off // 32, :, off % 32]
    return k, v


def attention(q, k, v, k_cache, v_cache, table, ctx_len, masks, n_nodes, scale, dtype):
    """(out, bound): the exact outputs [B][n][Hq][D] and how far a correct
    kernel of this precision may be from each.

    The bound adds up, per output, with A = sum p |v| / sum p:
      - the probabilities' rounding to `dtype` (at most UNIT of each) and the
        rounding of the output itself;
      - the scores' error d: fp32 dots of D products err by at most D 2^-24 of
        their absolute sum, their scaling and exponent by a few 2^-24 more; it
        moves every p by e^d, hence the output by at most 2 d A;
      - the fp32 sums over T positions: T 2^-24 of A each;
      - fp16 only: probabilities below 2^-14 of the maximum lose bits, at most
        2^-25 each, hence T 2^-25 max |v| over a sum that is at least 1."""
    B, n, Hq, D = q.shape
    H, page = k.shape[2], k_cache.shape[2]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        ctx = min(max(int(ctx_len[b]), 0), table.shape[1] * page)
        nodes = n if n_nodes is None else min(max(int(n_nodes[b]), 0), n)
        for h in range(H):
            kc, vc = cached_rows(k_cache, v_cache, table[b], h, ctx, page)
            for i in range(nodes):
                bits = (1 << (i + 1)) - 1 if masks is None else int(masks[b, i])
                see = [j for j in range(nodes) if bits >> j & 1]
                kk, vv = np.concatenate([kc, k[b, see, h]]), np.concatenate([vc, v[b, see, h]])
                if not len(kk):
                    continue
                for hq in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    s = scale * (kk @ q[b, i, hq])
                    p = np.exp(s - s.max())
                    out[b, i, hq] = p @ vv / p.sum()
                    A = p @ np.abs(vv) / p.sum()
                    T = len(kk)
                    d = 2.0 ** -24 * (D + 8) * abs(scale) * (np.abs(kk) @ np.abs(q[b, i, hq])).max()
                    u = UNIT[dtype]
                    bound[b, i, hq] = (u + 2 * d + 2 * T * 2.0 ** -24) * A + u * np.abs(out[b, i, hq]) + 2.0 ** -24
                    if dtype == "f16":
                        bound[b, i, hq] += T * 2.0 ** -25 * np.abs(vv).max()
    return out, bound


def softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def verify(target, draft, tokens, parents, n_nodes, temperature, uniforms, noise):
    """(tokens, path, count, margin): the committed tokens and path, and for
    each sequence how near the closest decision on its way was to falling the
    other way (relative)."""
    B, n, V = target.shape
    out, paths = np.full((B, n), -1, np.int64), np.full((B, n), -1, np.int64)
    counts, margins = np.zeros(B, np.int64), np.full(B, np.inf)

    def parent(b, i):
        p = i - 1 if parents is None else int(parents[b, i])
        return p if 0 <= p < i else -1

    for b in range(B):
        nodes = n if n_nodes is None else min(max(int(n_nodes[b]), 0), n)
        if nodes == 0:
            continue
        temp = 1.0 if temperature is None else float(temperature[b])
        path = [0]
        while True:
            v = path[-1]
            row = target[b, v].astype(np.float64)
            kids = [c for c in range(1, nodes) if parent(b, c) == v]
            took, token = None, None
            if temp == 0:
                token = int(np.argmax(row))  # numpy: the first NaN, else the first of the largest
                took = next((c for c in kids if int(tokens[b, c]) == token), None)
            else:
                p = left = softmax(row / temp)
                total = 1.0
                for c in kids:
                    x = int(tokens[b, c])
                    q = np.zeros(V)
                    if draft is not None:
                        q = softmax(draft[b, v].astype(np.float64) / temp)
                    elif 0 <= x < V:
                        q[x] = 1.0
                    if 0 <= x < V:
                        a, z = float(uniforms[b, c]) * q[x], left[x] / total
                        if max(a, z) > 0:  # 0 against 0 is exact on both sides
                            margins[b] = min(margins[b], abs(a - z) / max(a, z))
                        if a < z:
                            took = c
                            break
                    # an unnormalised remainder and its sum: a sum of zero stays one
                    left = np.maximum(0.0, left / total - q) if total > 0 else np.zeros(V)
                    total = left.sum()
                if took is None:
                    if not (left > 0).any():
                        left = p
                    score = np.where(left > 0, left / noise[b].astype(np.float64), -1.0)
                    token = int(np.argmax(score))
                    best = np.sort(score)[-2:]
                    if V > 1 and best[0] > 0:
                        margins[b] = min(margins[b], 1 - best[0] / best[1])
            if took is None:
                break
            path.append(took)
        counts[b] = len(path)
        paths[b, :len(path)] = path
        out[b, :len(path)] = [int(tokens[b, c]) for c in path[1:]] + [token]
    return out, paths, counts, margins


def append(k, v, k_cache, v_cache, table, ctx_len, path, count):
    """The caches [L][P]... after the append, and the new lengths."""
    k_cache, v_cache = k_cache.copy(), v_cache.copy()
    L, B, n = k.shape[:3]
    P, page = k_cache.shape[1], k_cache.shape[3]
    cap = table.shape[1] * page
    lens = np.zeros(B, np.int64)
    for b in range(B):
        ctx = min(max(int(ctx_len[b]), 0), cap)
        cnt = n if count is None else min(max(int(count[b]), 0), n)
        lens[b] = min(ctx + cnt, cap)
        for i in range(cnt):
            row = i if path is None else int(path[b, i])
            pos = ctx + i
            if pos >= cap or not 0 <= row < n:
                continue
            pg, off = int(table[b, pos // page]), pos % page
            if 0 <= pg < P:
                k_cache[:, pg, :, off] = k[:, b, row]
                v_cache[:, pg, :, off // 32, :, off % 32] = v[:, b, row]
    return k_cache, v_cache, lens


def ancestor_masks(parents):
    """uint64 [B][n]: bit j of entry i set where j is i or one of its ancestors."""
    B, n = parents.shape
    m = np.zeros((B, n), np.uint64)
    for b in range(B):
        for i in range(n):
            up = int(parents[b, i])
            m[b, i] = (m[b, up] if 0 <= up < i else np.uint64(0)) | np.uint64(1 << i)
    return m


def random_trees(B, n, g, branch=4):
    parents = np.full((B, n), -1, np.int32)
    for b in range(B):
        kids = [0] * n
        for i in range(1, n):
            free = [x for x in range(i) if kids[x] < branch][-6:]
            p = free[int(g.integers(len(free)))]
            kids[p] += 1
            parents[b, i] = p
    return parents
