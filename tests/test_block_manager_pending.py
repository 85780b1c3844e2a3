"""Shortening a sequence while copies are queued: a copy into a block that would be freed
is refused, so that it cannot land in the block's next owner.  Host code: no GPU."""
import pytest

import oracle
from paged_kv_cache_122_gb300 import BlockManager, PagedKVError


def _forked():
    """Sequence 2 shares 1's partial block 1 and copies it on its next append."""
    bm, ref = BlockManager(8, 4), oracle.CowBlockManager(8, 4)
    bm.add_sequence(1)
    ref.new_sequence(1)
    bm.append_slots([1] * 6)
    for _ in range(6):
        ref.append_slot(1)
    bm.fork(1, 2)
    ref.fork(1, 2)
    assert bm.append_slots([2]).tolist() == [ref.append_slot(2)]
    return bm, ref


def test_a_block_that_a_copy_is_queued_for_is_not_freed():
    bm, ref = _forked()
    before = bm.export([1, 2], 4), bm.num_free_blocks()
    for keep in (4, 0):
        with pytest.raises(PagedKVError) as e:
            bm.truncate(2, keep)
        assert e.value.status == -12 and "queued copy" in str(e.value)
        with pytest.raises(RuntimeError):
            ref.truncate(2, keep)
        after = bm.export([1, 2], 4), bm.num_free_blocks()
        assert all((a == b).all() for a, b in zip(before[0], after[0])) and before[1] == after[1]
    # What keeps the block, and what frees others, goes on.
    bm.truncate(2, 5)
    bm.truncate(1, 4)
    ref.truncate(2, 5)
    ref.truncate(1, 4)
    pairs = bm.take_copies()
    assert pairs.tolist() == [list(p) for p in ref.take_copies()] == [[1, 2]]
    bm.truncate(2, 4)
    ref.truncate(2, 4)
    assert bm.blocks_in_use() == ref.blocks_in_use() == 1 and bm.num_free_blocks() == 7


def test_a_shared_destination_is_not_freed_by_one_owner():
    bm, _ = _forked()
    bm.fork(2, 3)                        # 3 holds the copy's destination too
    bm.truncate(2, 4)
    with pytest.raises(PagedKVError) as e:
        bm.truncate(3, 4)
    assert e.value.status == -12
    assert bm.take_copies().tolist() == [[1, 2]]
    bm.truncate(3, 4)
    assert bm.blocks_in_use() == 2       # 1's two blocks
