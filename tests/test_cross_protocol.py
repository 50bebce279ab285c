"""The protocol of the d = 64 backward over keys of another length (cross_model) ends and keeps every buffer intact in
random orders of its roles, for blocks of one iteration and of many; planted mistakes are caught. CPU only."""
import random

import pytest

from cross_model import simulate_bwd_cross


@pytest.mark.parametrize("counts", [[], [1], [1, 1, 1, 1, 1], [2, 1, 3], [4] * 9, [7, 7], [1, 5, 1, 2, 2, 1], [20]])
def test_protocol_ends_and_keeps_its_buffers(counts):
    for seed in range(60):
        assert simulate_bwd_cross(counts, 3, seed)


def test_random_block_lists():
    rnd = random.Random(1)
    for seed in range(150):
        assert simulate_bwd_cross([rnd.randint(1, 6) for _ in range(rnd.randint(1, 8))], 3, seed)


@pytest.mark.parametrize("mistake", [dict(acc_free=False), dict(kv_free_count=1), dict(acc_waits=False),
                                     dict(readout_first=False)])
def test_planted_mistakes_are_caught(mistake):
    caught = 0
    for seed in range(300):
        try:
            simulate_bwd_cross([2, 1, 3, 1, 2, 4], 3, seed, **mistake)
        except AssertionError:
            caught += 1
    assert caught > 0
