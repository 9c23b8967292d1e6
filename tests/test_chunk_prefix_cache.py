"""Chunk reservations beside prefix caching (CPU only): a row that holds its
prompt's blocks already must not lose them."""

import numpy as np
import pytest


@pytest.fixture(scope="module")
def pa(built_library):
    from paged_kv_cache_341_b200 import pa as mod
    return mod


def state(pool, tables, lens):
    refs, free = pool.pa_pool_export()
    return [x.tolist() for x in (refs, free, tables, lens)] + [pool.pa_pool_cached_blocks()]


@pytest.mark.parametrize("second,cached", [(list(range(40)), 32), (list(range(33)) + [7] * 31, 32),
                                           ([9] * 40, 0), (list(range(16)) + [3], 16)])
def test_chunks_over_blocks_held_ahead_are_refused(pa, second, cached):
    """From the cached length on, each block start would take a new block in place of the row's own."""
    pool = pa.Pool(16, 16)
    pool.pa_pool_enable_prefix_cache()
    tables, lens = np.full((2, 8), -1, np.int32), np.zeros(2, np.int32)
    assert pool.pa_seq_alloc_prompt(list(range(40)), tables[0]) == 0
    lens[0] = 40
    assert pool.pa_seq_alloc_prompt(second, tables[1]) == cached
    lens[1] = cached
    before = state(pool, tables, lens)
    for counts in ([0, len(second) - cached], [0, 1], [9, 1]):
        with pytest.raises(pa.PagedAttnError) as e:
            pool.pa_reserve_chunks(tables, lens, counts)
        assert e.value.status == pa.PA_ERR_INVALID and state(pool, tables, lens) == before
    # the way that works: the prompt's tokens go to their slots in the table, then the length is the prompt's
    lens[1] = len(second)
    slots, _, _ = pool.pa_reserve_chunks(tables, lens, [20, 20])
    assert slots.size == 40 and lens.tolist() == [60, len(second) + 20]
    for r in range(2):
        pool.pa_pool_free(tables[r, :-(-int(lens[r]) // 16)])
    assert pool.pa_pool_num_free() == 16 and pool.pa_pool_cached_blocks() == 0


def test_a_chunk_that_starts_no_block_is_reserved(pa):
    """Within the row's last block nothing is taken, and nothing lost."""
    pool = pa.Pool(8, 16)
    pool.pa_pool_enable_prefix_cache()
    table, lens = np.full((1, 4), -1, np.int32), np.zeros(1, np.int32)
    pool.pa_seq_alloc_prompt(list(range(20)), table[0])
    lens[0] = 20
    slots, pairs, updates = pool.pa_reserve_chunks(table, lens, [12])
    assert slots.tolist() == [int(table[0, 1]) * 16 + 4 + i for i in range(12)]
    assert len(pairs) == 0 and len(updates) == 0 and pool.pa_pool_num_free() == 6


def test_stale_entries_are_overwritten_without_prefix_caching(pa):
    """As pa_seq_reserve_slot does: what stands behind a row's length is not read."""
    pool = pa.Pool(8, 16)
    tables, lens = np.full((2, 4), -1, np.int32), np.zeros(2, np.int32)
    tables[0, 0] = pool.pa_pool_alloc(1)[0]
    lens[0] = 16
    tables[1] = tables[0, 0]                                      # stale: row 1 holds nothing
    pool.pa_reserve_chunks(tables, lens, [0, 17])
    assert tables[1].tolist() == [1, 2, 0, 0] and pool.pa_pool_num_free() == 5
