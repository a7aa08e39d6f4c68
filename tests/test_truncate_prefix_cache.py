"""A sequence cut short inside a block that the prefix cache knows: the block's
old hash must not find it once it can be written again (CPU only)."""
import pytest

from paged_kv_cache_468_b200 import BlockAllocator, PagedKVError, pagedkv


def registered(a, tokens):
    """A sequence of `tokens` with its full blocks in the prefix cache."""
    blocks, _ = a.new_seq_cached(tokens)
    hashes = a.block_hashes(tokens)
    for h, b in zip(hashes, blocks):
        a.cache_insert(h, b)
    return blocks, hashes


def test_a_tail_block_that_is_written_again_is_forgotten():
    a = BlockAllocator(16, 4)
    old = list(range(8))
    seq, _ = registered(a, old)
    a.truncate(seq, 6)
    kept = list(seq)
    assert a.append(seq, 6, 8) is None and seq == kept      # written in place: two other tokens behind the first six
    other, hits = a.new_seq_cached(old)
    assert hits == 1 and other[0] == seq[0] and other[1] != seq[1]
    # the block can be registered under what it holds now
    new = old[:6] + [90, 91]
    h = a.block_hashes(new)[1]
    a.cache_insert(h, seq[1])
    assert a.cache_lookup(h) == seq[1]


@pytest.mark.parametrize("new_len", [5, 6, 7])
def test_cut_within_the_last_block_of_the_table(new_len):
    a = BlockAllocator(16, 4)
    seq, hashes = registered(a, list(range(8)))
    a.truncate(seq, new_len)                                 # the table keeps its length
    assert len(seq) == 2
    a.append(seq, new_len, 8)
    assert a.cache_lookup(hashes[1]) == -1
    assert a.cache_lookup(hashes[0]) == seq[0]


def test_blocks_that_stay_full_stay_registered():
    a = BlockAllocator(16, 4)
    seq, hashes = registered(a, list(range(12)))
    first = list(seq)
    a.truncate(seq, 8)
    a.append(seq, 8, 9)
    other, hits = a.new_seq_cached(list(range(12)))
    assert other[:2] == first[:2] and hits >= 2
    # the released third block held its tokens until it was handed out again
    assert (hits == 3) == (first[2] not in seq)


def test_a_shared_tail_block_is_copied_and_stays_registered():
    a = BlockAllocator(16, 4)
    seq, hashes = registered(a, list(range(8)))
    fork = a.fork(seq)
    a.truncate(seq, 6)
    assert a.append(seq, 6, 8) == (fork[1], seq[1]) and seq[1] != fork[1]
    assert a.cache_lookup(hashes[1]) == fork[1]


def test_a_shared_tail_block_whose_other_owner_left_is_forgotten():
    a = BlockAllocator(16, 4)
    seq, hashes = registered(a, list(range(8)))
    fork = a.fork(seq)
    a.truncate(seq, 6)
    a.free(fork)
    assert a.append(seq, 6, 8) is None
    assert a.cache_lookup(hashes[1]) == -1
    a.free(seq)
    assert a.num_free == 16 and a.cache_lookup(hashes[1]) == -1


def test_errors_change_nothing():
    a = BlockAllocator(6, 4)
    seq, hashes = registered(a, list(range(8)))
    gone = a.new_seq(4)
    a.free(gone)
    for bad in ([seq[0], -1, seq[1]], [seq[0], 6, seq[1]], [seq[0], gone[0], seq[1]]):
        with pytest.raises(PagedKVError) as e:
            a.truncate(bad, 6)                               # the block that would be the tail is not in use
        assert e.value.status == pagedkv.ERR_OUT_OF_RANGE and len(bad) == 3
    with pytest.raises(PagedKVError):
        a.truncate([seq[0], seq[1], gone[0]], 6)             # a released one that is free already
    assert a.num_free == 4 and a.cache_lookup(hashes[1]) == seq[1]
    # a growth that the pool has no blocks for forgets nothing either
    b = BlockAllocator(2, 4)
    seq, hashes = registered(b, list(range(8)))
    with pytest.raises(PagedKVError) as e:
        b.append(seq, 6, 16)
    assert e.value.status == pagedkv.ERR_OOM
    assert b.cache_lookup(hashes[1]) == seq[1]
