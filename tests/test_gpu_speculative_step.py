"""The example's speculative step: the operators run together as a user would
run them, and what they leave in the cache is what a plain pass leaves."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
E = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(E)


def _fill(model, cache, tokens):
    for at in range(0, tokens.shape[1], 64):
        _, keys, values = model.forward(tokens[:, at:at + 64].contiguous(), cache)
        cache.append(keys, values)


@pytest.mark.parametrize("nodes,kind", [(12, "tree"), (5, "chain")])
def test_committed_cache_is_that_of_the_committed_tokens(nodes, kind):
    """Some speculative steps, then the committed tokens once more, one after
    the other as a prompt: the same lengths, the same first-layer keys and
    values bit for bit (the projection's rows do not depend on their
    neighbours), and the second layer's within the rounding of the attention
    in between (2^-8 of values of size about 1, a few roundings)."""
    B, prompt_len, steps = 3, 37, 5
    model = E.Model(seed=3)
    g = torch.Generator(device=model.device)
    g.manual_seed(7)
    prompt = torch.randint(0, model.vocab, (B, prompt_len), generator=g, device=model.device, dtype=torch.int32)
    cache = E.Cache(model, B, prompt_len + steps * nodes)
    _fill(model, cache, prompt[:, :-1])
    tree = E.Tree([-1] + [(i - 1) // 3 if kind == "tree" else i - 1 for i in range(1, nodes)], B, model.device)
    root = prompt[:, -1]
    said = [prompt[b].tolist() for b in range(B)]
    for _ in range(steps):
        out, count = E.step(model, cache, tree, root, g)
        assert count.min().item() >= 1 and count.max().item() <= nodes
        for b, c in enumerate(count.tolist()):
            got = out[b].tolist()
            assert all(0 <= t < model.vocab for t in got[:c]) and all(t == -1 for t in got[c:])
            said[b] += got[:c]
        root = out.gather(1, (count.long() - 1)[:, None])[:, 0]
    # the last token of each sequence is the next root: not in the cache yet
    assert cache.lens.tolist() == [len(s) - 1 for s in said]
    for b in range(B):
        tokens = torch.tensor([said[b][:-1]], dtype=torch.int32, device=model.device)
        plain = E.Cache(model, 1, tokens.shape[1])
        _fill(model, plain, tokens)
        assert plain.lens.tolist() == [tokens.shape[1]]
        for t in range(tokens.shape[1]):
            mine, theirs = int(cache.table[b, t // 32]), int(plain.table[0, t // 32])
            k = cache.k[:, mine, :, t % 32], plain.k[:, theirs, :, t % 32]
            v = cache.v[:, mine, :, 0, :, t % 32], plain.v[:, theirs, :, 0, :, t % 32]
            for x, y in (k, v):
                assert torch.equal(x[0], y[0]), (b, t)
                assert (x[1].float() - y[1].float()).abs().max().item() <= 8 * 2.0 ** -8 * max(
                    1.0, y[1].float().abs().max().item()), (b, t)
