"""Rows of a tree attention call against each other: the bits of a row do not
depend on what its neighbours in the same matrix tile hold or see.

The contexts are long enough for every wave to fold several steps before the
nodes': the running maximum then moves within a wave's run, at steps that differ
from row to row."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq", [(64, 64), (128, 32), (256, 16)])
def test_a_neighbours_query_changes_nothing(D, Hq, dtype):
    """One head of one node asks for much larger scores: its maximum moves at
    other steps than those of the heads beside it."""
    n, L = 16, 16 * 520
    for head in (3, Hq - 1):
        c = Case(600 + D, dtype, n, Hq, 1, D, 64, [L], mask="tree")
        want = c.run()
        c.q[0, 5, head] *= 24.0
        got = c.run()
        keep = torch.ones(1, n, Hq, dtype=torch.bool)
        keep[0, 5, head] = False
        assert not torch.equal(got[~keep], want[~keep])
        assert torch.equal(_bits(got[keep]), _bits(want[keep]))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("what", [40.0, float("inf")])
def test_a_node_that_others_see_changes_nothing(what, dtype):
    """Large and infinite keys of a node that only some rows of a tile see."""
    n, L = 64, 16384
    c = Case(700, dtype, n, 8, 2, 64, 64, [L, 40], mask="tree")
    want = c.run()
    bad = n - 3
    sees = torch.from_numpy((c.masks >> np.uint64(bad)) & np.uint64(1) == 1)
    c.k[:, bad] *= what
    got = c.run()
    assert not torch.equal(got[sees], want[sees])
    assert torch.equal(_bits(got[~sees]), _bits(want[~sees]))
