"""The protocol of the shared prefix's kernel (prefix_model) ends and keeps every buffer intact in random orders of its
roles, with one and two tiles of query rows, warps without rows and two to six raw tiles in flight; planted mistakes are
caught. CPU only."""
import pytest

from prefix_model import simulate_prefix

DEAD = {1: [(), ((0, 3),), ((0, 1), (0, 2), (0, 3))], 2: [(), ((1, 2), (1, 3)), ((1, 1), (1, 2), (1, 3))]}


@pytest.mark.parametrize("tiles,raw", [(2, 2), (2, 4), (1, 4), (1, 6)])
@pytest.mark.parametrize("blocks", [1, 2, 3, 7, 16])
def test_protocol_ends_and_keeps_its_buffers(tiles, raw, blocks):
    for dead in DEAD[tiles]:
        for seed in range(25):
            assert simulate_prefix(blocks, tiles, raw, seed, dead)


@pytest.mark.parametrize("mistake", [dict(s_free=False), dict(k_empty=False), dict(v_empty=False), dict(raw_empty=False),
                                     dict(v_empty_count=1), dict(dead_wait=False, dead=((1, 2), (1, 3))), dict(pv_wait=False)])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(200):
        try:
            simulate_prefix(6, 2, 2, seed, **mistake)
        except AssertionError:
            caught += 1
    assert caught > 0
