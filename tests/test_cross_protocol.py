"""The plan of the backward over keys of another length covers every iteration once within its workspace, and the
protocol of the d = 64 backward over keys of another length (cross_model) ends and keeps every buffer intact in
random orders of its roles, for blocks of one iteration and of many; planted mistakes are caught. CPU only."""
import random

import pytest

from cross_model import item, plan, simulate_bwd_cross, slots


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


@pytest.mark.parametrize("sms", [1, 7, 152])
def test_plan_covers_every_iteration_once(sms):
    rnd = random.Random(sms)
    for _ in range(200):
        blocks, n_it = rnd.randint(1, 4 * sms), rnd.choice([1, 2, 3, 4, 20, 80, rnd.randint(1, 300)])
        valid = rnd.randint(0, blocks)
        full, parts, items = plan(valid, n_it, sms)
        room = slots(blocks, n_it, sms)
        launched = blocks + room if blocks > sms or room < blocks else room
        assert items <= launched and blocks <= launched and 1 <= parts <= max(n_it, 1)
        seen, used = {}, set()
        for a in range(items):
            rank, first, count, slot = item(full, parts, a, n_it)
            assert 0 <= rank < valid and count >= 1 and first + count <= n_it
            assert seen.get(rank, 0) == first  # a block's runs follow each other
            seen[rank] = first + count
            if slot >= 0:
                assert slot < room and slot not in used and slot // parts == rank - full
                used.add(slot)
        assert all(seen.get(r) == n_it for r in range(valid))
