"""Tree attention where almost all of the output comes from positions of very
small probability."""
import numpy as np
import pytest
import torch

from test_gpu_tree_attention import Case
from tree_ref import UNIT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("below", [4, 9, 12, 14, 16, 18])
def test_many_small_probabilities(below, D, dtype):
    """In every 32 tokens one has score 0 and value 0, the others score -below
    and value 2048: each output is 2048 * 31 e^-below / (1 + 31 e^-below), all
    of it from probabilities of e^-below of the largest.

    Bound, relative to the output: one rounding of each probability and one of
    the output (UNIT each); fp16 probabilities, kept 2^7 above the maximum's 1
    so that its 2^8 head room ends below 65504, err by at most 2^-32 of the
    maximum where they are subnormal; scores (exact products) times log2 e and
    their exponentials, 2^-24 of `below` and a few 2^-24; and the fp32 sums of
    640 terms, 640 * 2^-24 at most.  The output itself must not be subnormal."""
    n, L = 5, 640
    c = Case(800, dtype, n, 8, 2, D, 64, [L, L - 32], mask=None)
    c.scale = 1.0
    c.q[...] = 0
    c.q[..., 0] = 1.0
    c.k[...] = 0
    c.k[..., 0] = -512.0  # the nodes' own keys: nothing
    keys = torch.full((64, D), 0.0)
    keys[:, 0] = -float(below)
    keys[::32] = 0
    values = torch.full((2, D, 32), 2048.0)
    values[..., 0] = 0
    c.k_cache[...] = keys.to(c.k_cache.dtype)
    c.v_cache[...] = values.to(c.v_cache.dtype)
    p = np.exp(-float(below))
    want = 2048 * 31 * p / (1 + 31 * p)
    assert want > 2.0 ** -14
    bound = 2 * UNIT[dtype] + (2.0 ** -32 / p if dtype == "f16" else 0) + (2 * below + 8 + 640) * 2.0 ** -24
    got = c.run().to(torch.float64).numpy()
    assert np.abs(got / want - 1).max() <= bound, (np.abs(got / want - 1).max(), bound)


def test_probabilities_at_the_head_room_stay_finite():
    """Scores that rise by just under 2^8 after the first: probabilities of
    2^(8 + 7), and of their sum, are still finite in fp16."""
    c = Case(801, "f16", 2, 4, 1, 64, 32, [96], mask=None)
    c.scale = 1.0
    c.q[...] = 0
    c.q[..., 0] = 1.0
    c.k[...] = 0
    c.k_cache[...] = 0
    c.v_cache[...] = 60000.0
    c.k_cache[:, :, 8:, 0] = 5.54  # 5.54 log2 e = 7.99
    got = c.run()
    assert torch.isfinite(got).all()
    c.check(got)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_past_2_24(D):
    """Scores so large that neighbouring fp32 values are 2 apart: the choice to
    raise the base, and with it the bound on fp16 probabilities, must hold for
    the difference of two scores and not for a rounded sum.  Positions alternate
    by 128 between scores of s and s + 8 (in powers of two, s = 1.5 * 2^24), so
    that a wave meets both; values 1 and 2."""
    n, L = 64, 2048
    c = Case(802, "f16", n, 64, 1, D, 64, [L], mask=None)
    c.scale = 0.6931471824645996  # times log2 e = 1 in fp32
    c.q[...] = 0
    c.q[..., 0], c.q[..., 1] = 6144.0, 1.0
    c.k[...] = 0
    for page in range(L // 64):
        at, high = int(c.table[0, page]), page // 2 % 2
        c.k_cache[at], c.v_cache[at] = 0, 1.0 + high
        c.k_cache[at, ..., 0], c.k_cache[at, ..., 1] = 4096.0, 8.0 * high
    want = (1 + 2 * 256) / (1 + 256)
    got = c.run().to(torch.float64).numpy()
    # one rounding of the probabilities' weights (exact powers of two here) and one of the output
    assert np.abs(got / want - 1).max() <= 2 * UNIT["f16"], (got.min(), got.max(), want)
