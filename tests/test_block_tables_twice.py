"""A table that lists a block twice is refused by the block manager's calls for drafts and evictions (no GPU)."""
import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def pk():
    __graft_entry__.build()
    import paged_kv_decode_store_gb300 as pk
    return pk


def test_a_block_listed_twice(pk):
    """Released twice it would have fewer than no references, and be free while its key still finds it."""
    bm = pk.BlockManager(6, 4)
    table, _ = bm.allocate(list(range(9)))
    twice = [table[0], table[1], table[1]]
    for bad in (lambda: bm.reserve(9, 2, twice), lambda: bm.trim(list(range(9)), 9, twice + [table[2]]),
                lambda: bm.trim([0, 1, 2], 3, twice), lambda: bm.evict(4, twice), lambda: bm.evict(9, [table[0], table[2], table[0]])):
        with pytest.raises(pk.PkvdError):
            bad()
        assert bm.num_free() == 3 and [bm.ref_count(b) for b in table] == [1, 1, 1]
    bm.fork(table)                                           # held twice, but a sequence has it once
    with pytest.raises(pk.PkvdError):
        bm.trim([0, 1, 2], 3, twice)
    assert bm.num_free() == 3 and [bm.ref_count(b) for b in table] == [2, 2, 2]
    bm.release(table)
    grown, copy = bm.reserve(9, 5, table)                    # refused calls leave nothing behind
    assert len(grown) == 4 and copy is None and bm.trim(list(range(9)), 9, grown) == table
    assert bm.evict(4, table) == table[:1] and bm.num_free() == 5
