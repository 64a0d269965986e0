"""The example's speculative step with 8-bit decoder layers: what it leaves in
the cache is what a plain pass over the committed tokens leaves."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("speculative_step", os.path.join(ROOT, "examples", "speculative_step.py"))
E = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(E)


@pytest.mark.parametrize("nodes,kind", [(12, "tree"), (5, "chain")])
def test_committed_cache_is_that_of_the_committed_tokens(nodes, kind):
    """The first layer's keys, turned by the nodes' positions in their trees, and
    its values bit for bit: the products are exact and no row depends on its
    neighbours.  The second layer's follow the attention in between, whose sums
    run in another order over a tree than over a prompt.  Relative to the size of
    what they give: four bfloat16 roundings on the way (attention, two products,
    the keys and values themselves), 2^-8 each, and 8-bit codes that such a
    difference moves by one, 1/127 of a row's largest, which is about four times
    its mean size: 4/127, with 1 in 16 codes allowed to move, whose norm is
    sqrt(1/16) of all codes'.  That share is an allowance and no proof; a wrong
    position, row or mask differs by about the whole size."""
    B, prompt_len, steps = 3, 37, 4
    model = E.Int8Model(seed=3)
    g = torch.Generator(device=model.device)
    g.manual_seed(7)
    prompt = torch.randint(0, model.vocab, (B, prompt_len), generator=g, device=model.device, dtype=torch.int32)

    def fill(cache, tokens):
        for at in range(0, tokens.shape[1], 64):
            _, keys, values = model.forward(tokens[:, at:at + 64].contiguous(), cache)
            cache.append(keys, values)
    cache = E.Cache(model, B, prompt_len + steps * nodes)
    fill(cache, prompt[:, :-1])
    tree = E.Tree([-1] + [(i - 1) // 3 if kind == "tree" else i - 1 for i in range(1, nodes)], B, model.device)
    root, said = prompt[:, -1], [prompt[b].tolist() for b in range(B)]
    for _ in range(steps):
        out, count = E.step(model, cache, tree, root, g)
        for b, c in enumerate(count.tolist()):
            said[b] += out[b].tolist()[:c]
        root = out.gather(1, (count.long() - 1)[:, None])[:, 0]
    assert cache.lens.tolist() == [len(s) - 1 for s in said]
    for b in range(B):
        tokens = torch.tensor([said[b][:-1]], dtype=torch.int32, device=model.device)
        plain = E.Cache(model, 1, tokens.shape[1])
        fill(plain, tokens)
        n = tokens.shape[1]
        for c, one in ((cache.k, plain.k), (cache.v.transpose(-1, -2).flatten(3, 4), plain.v.transpose(-1, -2).flatten(3, 4))):
            mine = c[:, cache.table[b].long()].transpose(1, 2).flatten(2, 3)[:, :, :n].float()
            theirs = one[:, plain.table[0].long()].transpose(1, 2).flatten(2, 3)[:, :, :n].float()
            assert torch.equal(mine[0], theirs[0]) and mine[0].abs().max() > 0
            assert (mine[1] - theirs[1]).norm() <= (4 * 2.0 ** -8 + 4.0 / 127 * (1 / 16) ** 0.5) * theirs[1].norm()
