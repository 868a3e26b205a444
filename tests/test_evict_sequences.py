"""The block manager's side of an eviction of several sequences: the new tables of
a batch never name a block that its old tables read.  Host only."""
import numpy as np
import pytest


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_224_gb300 import build
    build.build()


def manager(blocks, bs, cache, lens):
    import paged_kv_cache_224_gb300 as pa
    m = pa.BlockManager(blocks, bs, prefix_cache=cache)
    for s, n in enumerate(lens):
        m.add_sequence(s, [1000 * s + j for j in range(n)])
    return m


def state(m, seqs):
    return [(m.seq_len(s), list(m.block_table(s))) for s in seqs], m.stats()["used_blocks"]


@pytest.mark.parametrize("cache", [True, False])
@pytest.mark.parametrize("spare", [0, 1, 64])
@pytest.mark.parametrize("lens", [[200] * 8, [160, 160], [40, 200, 0, 64, 65, 63, 1]])
def test_a_batch_takes_no_block_that_it_still_reads(cache, spare, lens):
    bs, keep = 16, 64
    old_n = sum(-(-n // bs) for n in lens)
    new_n = sum(-(-min(n, keep) // bs) for n in lens)
    m = manager(old_n + new_n + spare, bs, cache, lens)     # spare 0: every block is in use afterwards
    seqs = range(len(lens))
    old = [set(map(int, m.block_table(s))) for s in seqs]
    m.evict_sequences(list(seqs), keep)
    new = [list(map(int, m.block_table(s))) for s in seqs]
    flat = [b for r in new for b in r]
    assert len(set(flat)) == len(flat) == new_n and not set(flat) & set().union(*old)
    assert [m.seq_len(s) for s in seqs] == [min(n, keep) for n in lens]
    assert all(m.refcount(b) == 1 for b in flat)
    assert m.stats()["used_blocks"] == new_n


@pytest.mark.parametrize("cache", [True, False])
def test_all_or_nothing(cache):
    import paged_kv_cache_224_gb300 as pa
    lens, bs = [160, 160, 30], 16                           # 22 blocks; 4 + 4 + 2 new ones
    m = manager(31, bs, cache, lens)
    before = state(m, range(3))
    for ids, keep, status in (([0, 1, 2], 64, -8),          # one block short
                              ([0, 1, 0], 16, -1), ([0, 7], 16, -1), ([0, 1], -1, -3)):
        with pytest.raises(pa.PAError) as e:
            m.evict_sequences(ids, keep)
        assert e.value.status == status
        assert state(m, range(3)) == before
    m.evict_sequences([], 16)
    assert state(m, range(3)) == before
    m.evict_sequences([0, 1], 64)
    m.evict_sequences([2], 0)
    assert [m.seq_len(s) for s in range(3)] == [64, 64, 0] and m.stats()["used_blocks"] == 8
    with pytest.raises(ValueError):
        m.evict_sequences([[0, 1]], 16)


def test_shared_blocks_and_growth_after_it():
    m = manager(64, 4, True, [18])
    m.fork(0, 1)
    m.fork(0, 2)
    shared = list(m.block_table(0))
    m.evict_sequences(np.array([0, 2]), 7)
    tables = [list(m.block_table(s)) for s in range(3)]
    assert tables[1] == shared and not set(tables[0]) & set(shared) and not set(tables[0]) & set(tables[2])
    # they go on in their own blocks, without a copy, and never join the prefix tree
    slots = [m.append_token(2, j) for j in range(6)]
    assert slots[0] == (tables[2][1] * 4 + 3, None) and all(pair is None for _, pair in slots)
    for s in range(3):
        m.free_sequence(s)
    assert m.stats()["cached_free_blocks"] == 4 and m.stats()["used_blocks"] == 0


def test_what_the_readme_shows():
    # the lines of the README's bounded cache, with the device calls left out
    seqs, keep, block_size = [0, 1, 2, 3], 64, 16
    bm = manager(200, block_size, True, [200, 40, 130, 64])
    old = bm.tables(seqs)
    bm.evict_sequences(seqs, keep)
    new = bm.tables(seqs, -(-keep // block_size))
    assert new.shape == (4, 4) and not set(new[new >= 0]) & set(old[old >= 0])
