"""The host block manager's compaction of the sequences that one eviction takes (CPU): no block that one of them is
handed may be one that another's tokens still lie in, whatever the pool's order."""
import numpy as np
import pytest

import paged_kv_cache_121_gb300 as pa


def tables(bm, seqs):
    return [bm.block_table(s) for s in seqs]


def flat(rows):
    return [b for row in rows for b in row]


def test_new_tables_meet_no_old_one_of_the_group():
    bm = pa.BlockManager(30, 16, reserve_null_block=False)
    seqs = [3, 1, 7]
    for s in seqs:
        bm.allocate(s, 96)                         # 6 blocks each
    old = tables(bm, seqs)
    new = bm.compact_group(seqs, [48, 96, 1])
    assert [len(t) for t in new] == [3, 6, 1] and new == tables(bm, seqs)
    assert not set(flat(new)) & set(flat(old)) and len(set(flat(new))) == 10
    assert [bm.num_tokens(s) for s in seqs] == [48, 96, 1]
    assert flat(new) == list(range(18, 28))        # taken from the front, sequence after sequence
    assert bm.free_list() == flat(old) + [28, 29]  # released to the front, in the tables' order


@pytest.mark.parametrize("seed", range(20))
def test_random_pools_forks_and_groups(seed):
    rng = np.random.default_rng(seed)
    bs = int(rng.integers(1, 20))
    bm = pa.BlockManager(200, bs, free_order=rng.permutation(200))
    live = list(range(int(rng.integers(1, 7))))
    for s in live:
        bm.allocate(s, int(rng.integers(0, 10 * bs)))
    for s in live[: len(live) // 2]:
        bm.fork(s, 100 + s)
    everything = live + [100 + s for s in live[: len(live) // 2]]
    group = [int(s) for s in rng.permutation(everything)[: int(rng.integers(0, len(everything) + 1))]]
    before = {s: bm.block_table(s) for s in everything}
    tokens = [int(rng.integers(0, bm.num_tokens(s) + 1)) for s in group]
    new = bm.compact_group(group, tokens)
    held = [b for s in everything for b in before[s]]
    assert not set(flat(new)) & set(held) and len(set(flat(new))) == len(flat(new))
    for s in everything:
        if s in group:
            i = group.index(s)
            assert bm.block_table(s) == new[i] and bm.num_tokens(s) == tokens[i] and len(new[i]) == -(-tokens[i] // bs)
        else:
            assert bm.block_table(s) == before[s]   # a fork outside the group keeps its blocks
    now = [b for s in everything for b in bm.block_table(s)]
    for b in range(200):
        assert bm.refcount(b) == now.count(b)
    assert sorted(bm.free_list()) == [b for b in range(200) if b not in now]


def test_refusals_change_nothing():
    bm = pa.BlockManager(21, 16)                   # 20 usable
    for s in (0, 1, 2):
        bm.allocate(s, 70)                         # 5 each
    bm.fork(0, 9)
    state = lambda: (tables(bm, (0, 1, 2, 9)), bm.free_list(), bm.stats())  # noqa: E731
    before = state()
    for seqs, tokens, status in (([0, 1], [48, 49], pa.PA_ERR_OUT_OF_BLOCKS), ([0, 0], [1, 1], pa.PA_ERR_INVALID_ARG),
                                 ([0, 5], [1, 1], pa.PA_ERR_NOT_FOUND), ([0, 1], [16, 71], pa.PA_ERR_INVALID_ARG),
                                 ([2, 1], [16, -1], pa.PA_ERR_INVALID_ARG)):
        with pytest.raises(pa.PAError) as e:
            bm.compact_group(seqs, tokens)
        assert e.value.status == status and state() == before
    for seqs, tokens in (([0, 1], [1]), ([0], [[1]])):
        with pytest.raises(ValueError):
            bm.compact_group(seqs, tokens)
    assert bm.compact_group([], []) == [] and state() == before
    bm.enable_swap(8)
    bm.swap_out([1])
    before = state()
    with pytest.raises(pa.PAError) as e:
        bm.compact_group([2, 1], [1, 1])
    assert e.value.status == pa.PA_ERR_INVALID_ARG and state() == before


def test_a_short_table_is_refused_and_says_how_long_it_has_to_be():
    import ctypes
    bm = pa.BlockManager(21, 16)
    bm.allocate(0, 40)
    bm.allocate(1, 40)
    lib, n = pa.load_library(), ctypes.c_int(0)
    ids, tokens, out = (ctypes.c_int64 * 2)(0, 1), (ctypes.c_int * 2)(33, 16), (ctypes.c_int32 * 4)()
    free = bm.free_list()
    assert lib.pa_bm_compact_group(bm._h, ids, 2, tokens, out, 3, ctypes.byref(n)) == pa.PA_ERR_INVALID_ARG
    assert n.value == 4 and bm.free_list() == free
    for bad in ((None, ids, 2, tokens, out, 4, ctypes.byref(n)), (bm._h, None, 2, tokens, out, 4, ctypes.byref(n)),
                (bm._h, ids, -1, tokens, out, 4, ctypes.byref(n)), (bm._h, ids, 2, None, out, 4, ctypes.byref(n)),
                (bm._h, ids, 2, tokens, None, 4, ctypes.byref(n)), (bm._h, ids, 2, tokens, out, 4, None)):
        assert lib.pa_bm_compact_group(*bad) == pa.PA_ERR_INVALID_ARG and bm.free_list() == free
    assert lib.pa_bm_compact_group(bm._h, ids, 2, tokens, out, 4, ctypes.byref(n)) == pa.PA_OK
    assert list(out) == bm.block_table(0) + bm.block_table(1)


def test_one_by_one_the_second_sequence_is_handed_the_first_ones_blocks():
    """Why a group has a call of its own: what a lone compaction releases is handed out next."""
    bm = pa.BlockManager(12, 16, reserve_null_block=False)
    for s in (0, 1):
        bm.allocate(s, 64)
    old = bm.block_table(0)
    bm.compact(0, 32)
    assert set(bm.compact(1, 32)) <= set(old)
