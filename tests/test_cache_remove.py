"""Blocks taken out of the prefix cache before their cells are rewritten in
place, as a compaction does (CPU only)."""
import pytest

from paged_kv_cache_468_b200 import BlockAllocator, PagedKVError, pagedkv


def registered(a, tokens):
    blocks, _ = a.new_seq_cached(tokens)
    for h, b in zip(a.block_hashes(tokens), blocks):
        a.cache_insert(h, b)
    return blocks


def test_rewritten_blocks_are_not_found():
    a = BlockAllocator(16, 4)
    tokens = list(range(12))
    seq = registered(a, tokens)
    a.cache_remove(seq[1:])                                  # cells 4 .. 11 are about to be compacted
    other, hits = a.new_seq_cached(tokens)
    assert hits == 1 and other[0] == seq[0] and not set(other[1:]) & set(seq)
    a.cache_remove(seq[1:])                                  # not registered: nothing to do
    a.cache_remove([])
    # what the blocks hold afterwards can be registered
    h = a.block_hashes(tokens[:4] + [7, 8, 9, 10])[1]
    a.cache_insert(h, seq[1])
    assert a.cache_lookup(h) == seq[1]


def test_a_released_block_becomes_free():
    a = BlockAllocator(3, 4)
    seq = registered(a, list(range(12)))
    hashes = a.block_hashes(list(range(12)))
    a.free(seq)
    a.cache_remove([seq[2], seq[0]])
    assert a.num_free == 3
    assert a.cache_lookup(hashes[0]) == -1 and a.cache_lookup(hashes[2]) == -1
    # the free ones are handed out before the one that is still cached
    taken = a.new_seq(8)
    assert set(taken) == {seq[0], seq[2]} and a.cache_lookup(hashes[1]) == seq[1]
    assert a.num_free == 0


def test_a_block_outside_the_pool_changes_nothing():
    a = BlockAllocator(4, 4)
    seq = registered(a, list(range(8)))
    hashes = a.block_hashes(list(range(8)))
    for bad in ([seq[0], 4], [seq[0], -1]):
        with pytest.raises(PagedKVError) as e:
            a.cache_remove(bad)
        assert e.value.status == pagedkv.ERR_OUT_OF_RANGE
    assert a.cache_lookup(hashes[0]) == seq[0]
    L = pagedkv.lib()
    assert L.pkv_alloc_cache_remove(None, None, 0) == pagedkv.ERR_INVALID_ARG
    assert L.pkv_alloc_cache_remove(a._h, None, 1) == pagedkv.ERR_INVALID_ARG
    assert L.pkv_alloc_cache_remove(a._h, None, -1) == pagedkv.ERR_INVALID_ARG
    assert L.pkv_alloc_cache_remove(a._h, None, 0) == pagedkv.OK
