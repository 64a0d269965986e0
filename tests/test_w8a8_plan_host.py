"""How the 8-bit products are laid out, on the host: that every tile is
computed once, that nothing is cut without room, and which forms the shapes of
the GPU tests reach."""
import random

import pytest

import block_quantized_gemm_amd as vq
import plan_host as H
import test_gpu_w8a8 as G

SHAPES = [(n, m, k) for n in (1, 16, 17, 33, 100, 300, 4093) for m in (1, 130, 5120, 17408) for k in (16, 1040, 17408)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("cus", [256, 304, 80, 1])
def test_every_tile_once(gated, cus):
    """Whole tiles and cut ones together are the grid's tiles; the cut ones'
    pieces are no more than the workgroups, which all of them run at once, nor
    than the chunks."""
    rng = random.Random(cus)
    shapes = SHAPES + [(rng.randint(1, 5000), rng.randint(1, 20000), 16 * rng.randint(1, 1200)) for _ in range(300)]
    for n, m, k in shapes:
        for room in (0, H.ROOM):
            p = H.plan(n, m, k, gated, room, cus)
            rows, cols = H.tiles(p, n, m, gated)
            rest = rows * cols - p.whole
            assert 0 <= rest and p.groups >= 1, (n, m, k, p)
            if room == 0 or rest == 0:
                assert rest == 0 and p.cuts == 0, (n, m, k, p)
            else:
                assert p.cuts >= 2 and rest * p.cuts <= p.groups, (n, m, k, p)
                assert p.cuts <= -(-k // (128 * p.wk)), (n, m, k, p)


def test_the_gpu_shapes_reach_every_form():
    """Each form with whole tiles, with cut tiles, and (for the large ones)
    with whole rounds and cut tiles behind them."""
    for shapes, gated in ((G.PLAIN, False), (G.GATED, True)):
        seen = {}
        for n, m, k in shapes:
            p = H.plan(n, m, k, gated)
            kind = "whole" if p.cuts == 0 else "cut" if p.whole == 0 else "both"
            seen.setdefault(p.form, set()).add(kind)
        assert sorted(seen) == list(range(H.lib().forms())), seen
        assert all("whole" in kinds and len(kinds) > 1 for kinds in seen.values()), seen


def test_weights_read_again_stay_in_the_caches():
    """Weights are loaded past the caches only where they are too large for
    them and are read by one row of tiles, or by two of 16 x 128, whatever the
    height of the form: 17 to 32 rows in 16 x 32 tiles are two rows of them."""
    big = [(17408, 17408), (8192, 17408), (17408, 8192), (40960, 4096), (5120, 65536)]
    seen = set()
    for gated in (False, True):
        for m, k in big + [(5120, 8192), (700, 17408)]:
            for n in (1, 9, 16, 17, 24, 32, 33, 40, 61, 64, 65, 100, 129, 256, 257, 2048):
                p = H.plan(n, m, k, gated)
                rows = H.tiles(p, n, m, gated)[0]
                large = m * k * (2 if gated else 1) >= 128 << 20
                assert p.past == (large and (rows == 1 or (rows == 2 and (p.rows, p.feats) == (16, 128)))), (n, m, k, p)
                seen.add((large, min(rows, 3), p.rows, p.past))
    assert {(True, 1, 16, 1), (True, 1, 64, 1), (True, 2, 16, 0), (True, 2, 16, 1), (False, 1, 16, 0)} <= seen, seen
    assert not H.plan(17, 8192, 17408).past and H.plan(16, 8192, 17408).past and H.plan(61, 17408, 5120, True).past


def test_bytes_used_of_a_workspace():
    """As the library answers (it takes 256 compute units where there is no
    device): 0 exactly where nothing is cut, never more than what is asked for."""
    for gated in (False, True):
        for n, m, k in SHAPES + (G.GATED if gated else G.PLAIN):
            used, p = vq.w8a8_workspace_used(n, m, k, gated), H.plan(n, m, k, gated)
            rows, cols = H.tiles(p, n, m, gated)
            pieces = (rows * cols - p.whole) * p.cuts * p.rows * p.feats * 4
            assert used == (H.lib().counter_bytes() + pieces if p.cuts else 0), (n, m, k, p)
            assert used <= vq.w8a8_workspace_bytes(n)
    for bad in ((0, 16, 16), (1, 0, 16), (1, 16, 24), (1, 16, 0), ((1 << 24) + 1, 16, 16), (1, 16, 131072)):
        assert vq.w8a8_workspace_used(*bad) == 0
