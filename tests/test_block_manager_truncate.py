"""Shortening a sequence (rejected drafts): the library's block manager against the
oracle's, step by step, and its refusals.  Host code: no GPU."""
import numpy as np
import pytest

import oracle
from paged_kv_cache_122_gb300 import BlockManager, PagedKVError


def _table(bm, sid):
    nb = bm.sequence_info(sid)[1]
    return [int(x) for x in bm.export([sid], max(nb, 1))[0][0][:nb]]


@pytest.mark.parametrize("B", [1, 8, 16])
def test_random_drafts_match_the_oracle(B):
    rng = np.random.default_rng(B)
    bm, ref = BlockManager(40, B), oracle.CowBlockManager(40, B)
    bm.add_sequence(0)
    ref.new_sequence(0)
    alive, nxt = [0], 1
    for step in range(300):
        s = int(rng.choice(alive))
        n = int(rng.integers(1, 2 * B + 2))
        if bm.num_free_blocks() > n // B + 2:
            slots = bm.append_slots([s] * n)
            assert slots.tolist() == [ref.append_slot(s) for _ in range(n)]
            assert bm.take_copies().tolist() == [list(p) for p in ref.take_copies()]
        kept = int(rng.integers(0, ref.lengths[s] + 1)) if rng.random() < 0.2 else max(0, ref.lengths[s] - int(rng.integers(0, n + 1)))
        bm.truncate(s, kept)
        ref.truncate(s, kept)
        if rng.random() < 0.1 and len(alive) < 5:
            bm.fork(s, nxt)
            ref.fork(s, nxt)
            alive.append(nxt)
            nxt += 1
        for a in alive:
            assert _table(bm, a) == ref.tables[a] and bm.sequence_info(a)[0] == ref.lengths[a]
        assert bm.blocks_in_use() == ref.blocks_in_use() and bm.num_free_blocks() == len(ref.free)


def test_a_shared_block_outlives_the_sequence_that_drops_it():
    bm = BlockManager(8, 4)
    bm.add_sequence(1)
    bm.append_slots([1] * 6)
    bm.fork(1, 2)
    bm.truncate(2, 4)
    assert bm.blocks_in_use() == 2 and _table(bm, 2) == _table(bm, 1)[:1]
    bm.truncate(1, 4)
    assert bm.blocks_in_use() == 1
    bm.truncate(1, 0)
    assert _table(bm, 1) == [] and bm.blocks_in_use() == 1
    bm.truncate(2, 0)
    assert bm.blocks_in_use() == 0 and bm.append_slots([1]).shape == (1,)


def test_refusals():
    bm = BlockManager(8, 4)
    bm.add_sequence(1)
    bm.append_slots([1] * 5)
    for n in (-1, 6, 1 << 40):
        with pytest.raises(PagedKVError) as e:
            bm.truncate(1, n)
        assert e.value.status == -2
    with pytest.raises(PagedKVError) as e:
        bm.truncate(7, 0)
    assert e.value.status == -9
    assert bm.sequence_info(1) == (5, 2)
