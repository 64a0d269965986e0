"""Speculative decoding with a tree of drafted tokens, on random weights:

    python examples/speculative_step.py [--steps 8] [--batch 4] [--nodes 16]

A small transformer (attention and a Q4_0 projection on each side of it, no
MLP) generates with a bigram table as its drafter.  One step, all of it on the
device and without a host synchronisation:

  draft    a tree per sequence, each node's children drawn from the drafter's row
  per layer
    vq.gemm_q4_0        queries, keys and values of every node (one fused matrix)
    vq.tree_attention   over the sequence's cache and the node's ancestors
    vq.gemm_q4_0        back to the hidden width, added to the residual
  vq.gemm_q4_0          logits of every node
  vq.tree_verify        the accepted path and the next token, from random numbers
  vq.kv_append          the accepted nodes' keys and values, all layers at once
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_quantized_gemm_amd as vq  # noqa: E402


class Model:
    """Random Q4_0 weights of a small target and the drafter's bigram logits."""

    def __init__(self, layers=2, hidden=512, q_heads=8, kv_heads=2, dim=64, vocab=512, seed=0, device="cuda"):
        self.layers, self.hidden, self.vocab = layers, hidden, vocab
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        self.device = torch.device(device)
        g = torch.Generator().manual_seed(seed)

        def q4_0(m, k):  # codes uniform, scales so that a row of unit inputs gives about a unit output
            codes = torch.randint(0, 256, (m, k // 2), generator=g, dtype=torch.uint8)
            scales = torch.full((m, k // 32), 0.21 / k ** 0.5).to(torch.float16)
            return codes.to(self.device), scales.to(self.device)

        self.qkv = [q4_0((q_heads + 2 * kv_heads) * dim, hidden) for _ in range(layers)]
        self.back = [q4_0(hidden, q_heads * dim) for _ in range(layers)]
        self.head = q4_0(vocab, hidden)
        self.embedding = torch.randn(vocab, hidden, generator=g).to(torch.bfloat16).to(self.device)
        self.bigram = (1.5 * torch.randn(vocab, vocab, generator=g)).to(torch.bfloat16).to(self.device)

    def _matmul(self, w, x):
        out = torch.empty(x.shape[0], w[0].shape[0], dtype=torch.bfloat16, device=x.device)
        return vq.gemm_q4_0(w[0], w[1], x, out)

    def forward(self, tokens, cache, tree_mask=None):
        """(logits [B][n][vocab], keys, values [layers][B][n][kv_heads][dim])
        of n nodes per sequence over what the cache holds."""
        B, n = tokens.shape
        x = self.embedding[tokens.long().view(-1)]
        keys = torch.empty(self.layers, B, n, self.kv_heads, self.dim, dtype=x.dtype, device=x.device)
        values = torch.empty_like(keys)
        widths = [self.q_heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim]
        for i in range(self.layers):
            rows = self._matmul(self.qkv[i], x).view(B, n, -1)
            q, k, v = (t.unflatten(-1, (-1, self.dim)) for t in torch.split(rows, widths, dim=-1))
            seen = vq.tree_attention(q, k, v, cache.k[i], cache.v[i], cache.table, cache.lens, tree_mask=tree_mask)
            x = x + self._matmul(self.back[i], seen.view(B * n, -1))
            keys[i], values[i] = k, v
        return self._matmul(self.head, x.contiguous()).view(B, n, -1), keys, values


class Cache:
    """Pages of all layers; each sequence owns `capacity` tokens' worth of them."""

    def __init__(self, model, batch, capacity, page=32):
        per = -(-capacity // page)
        shape = (model.layers, batch * per, model.kv_heads)
        self.k = torch.zeros(*shape, page, model.dim, dtype=torch.bfloat16, device=model.device)
        self.v = torch.zeros(*shape, page // 32, model.dim, 32, dtype=torch.bfloat16, device=model.device)
        order = torch.randperm(batch * per, generator=torch.Generator().manual_seed(batch))
        self.table = order.to(torch.int32).view(batch, per).to(model.device)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=model.device)

    def append(self, keys, values, path=None, count=None):
        self.lens = vq.kv_append(keys, values, self.k, self.v, self.table, self.lens, path=path, count=count)


class Tree:
    """A fixed shape of draft tree: parents [n] with parents[0] = -1 and every
    parent before its children."""

    def __init__(self, parents, batch, device):
        masks = []
        for i, up in enumerate(parents):
            masks.append((masks[up] if i else 0) | 1 << i)
        as_int64 = [m - (1 << 64) if m >> 63 else m for m in masks]
        self.up = list(parents)
        self.parents = torch.tensor(parents, dtype=torch.int32, device=device).repeat(batch, 1)
        self.mask = torch.tensor(as_int64, dtype=torch.int64, device=device).repeat(batch, 1)


def draft(model, tree, root, generator):
    """(tokens [B][n], drafter logits [B][n][vocab]): each node's children are
    independent draws from its row."""
    B, n = tree.parents.shape
    tokens = torch.zeros(B, n, dtype=torch.int32, device=model.device)
    logits = torch.empty(B, n, model.vocab, dtype=torch.bfloat16, device=model.device)
    tokens[:, 0] = root
    for i in range(n):
        if i > 0:
            row = logits[:, tree.up[i]].float()
            noise = torch.empty_like(row).exponential_(generator=generator)
            tokens[:, i] = (row - torch.log(noise)).argmax(-1).to(torch.int32)
        logits[:, i] = model.bigram[tokens[:, i].long()]
    return tokens, logits


def step(model, cache, tree, root, generator):
    """One speculative step from the last committed token of each sequence.
    Returns (tokens [B][n], count [B]): the committed tokens, -1 past count."""
    B, n = tree.parents.shape
    tokens, drafted = draft(model, tree, root, generator)
    logits, keys, values = model.forward(tokens, cache, tree.mask)
    uniforms = torch.rand(B, n, device=model.device, generator=generator)
    noise = torch.empty(B, model.vocab, device=model.device).exponential_(generator=generator)
    out, path, count = vq.tree_verify(logits, drafted, tokens, uniforms, noise, parents=tree.parents)
    cache.append(keys, values, path=path, count=count)
    return out, count


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--nodes", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=40)
    args = ap.parse_args()
    model = Model()
    cache = Cache(model, args.batch, args.prompt + args.steps * args.nodes)
    g = torch.Generator(device=model.device)
    g.manual_seed(1)
    # the prompt, 64 tokens at a time as a chain; its last token is the first tree's root
    prompt = torch.randint(0, model.vocab, (args.batch, args.prompt), generator=g, device=model.device,
                           dtype=torch.int32)
    for at in range(0, args.prompt - 1, 64):
        _, keys, values = model.forward(prompt[:, at:min(at + 64, args.prompt - 1)].contiguous(), cache)
        cache.append(keys, values)
    tree = Tree([-1] + [(i - 1) // 2 for i in range(1, args.nodes)], args.batch, model.device)
    root = prompt[:, -1]
    for s in range(args.steps):
        out, count = step(model, cache, tree, root, g)
        root = out.gather(1, (count.long() - 1)[:, None])[:, 0]
        print("step %d: committed %s" % (s, [out[b, :c].tolist() for b, c in enumerate(count.tolist())]))
    print("lengths %s" % cache.lens.tolist())


if __name__ == "__main__":
    main()
