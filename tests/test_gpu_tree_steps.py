"""Several verification steps in a row on a pool with prefix caching: drafts
appended, written, masked, accepted, compacted and cut off, committed blocks
registered, a sequence rolled back and continued with other tokens.  K/V are a
function of (token, position), so every cell that a table or the prefix cache
gives can be checked for what it has to hold."""
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from tests import tree_util as tu

pytestmark = pytest.mark.gpu

Hkv, D, BS, LAYERS, POOL = 2, 64, 16, 2, 96


def _kv(tokens, positions, layer):
    """K and V [n, Hkv, D] of tokens at positions (bf16-exact whole numbers)."""
    t = torch.tensor(tokens, dtype=torch.float32)[:, None, None]
    p = torch.tensor(positions, dtype=torch.float32)[:, None, None]
    d = torch.arange(Hkv * D, dtype=torch.float32).view(1, Hkv, D)
    k = (t * 7 + p * 3 + d + layer * 11) % 127
    return k.to(torch.bfloat16), (126 - k).to(torch.bfloat16)


class _Server:
    def __init__(self):
        self.alloc = pkv.BlockAllocator(POOL, BS, shuffle_seed=9)
        self.k = [torch.zeros(POOL, BS, Hkv, D, dtype=torch.bfloat16).cuda() for _ in range(LAYERS)]
        self.v = [torch.zeros(POOL, BS, Hkv, D, dtype=torch.bfloat16).cuda() for _ in range(LAYERS)]

    def write(self, table, cells, tokens, positions):
        if not cells:
            return
        slots = torch.tensor([table[c // BS] * BS + c % BS for c in cells]).cuda()
        for i in range(LAYERS):
            k, v = _kv(tokens, positions, i)
            pkv.kv_cache_write(k.cuda(), v.cuda(), slots, self.k[i], self.v[i])

    def grow(self, table, old, new):
        pair = self.alloc.append(table, old, new)
        if pair:
            m = torch.tensor([pair], dtype=torch.int32).cuda()
            for i in range(LAYERS):
                pkv.copy_blocks(self.k[i], self.v[i], self.k[i], self.v[i], m)

    def start(self, tokens):
        table, hits = self.alloc.new_seq_cached(tokens)
        rest = list(range(hits * BS, len(tokens)))
        self.write(table, rest, [tokens[c] for c in rest], rest)
        self.register(table, tokens)
        return table

    def register(self, table, tokens):
        for h, b in zip(self.alloc.block_hashes(tokens), table):
            self.alloc.cache_insert(h, b)

    def holds(self, table, tokens):
        """The table's cells hold the K/V of these tokens."""
        n = len(tokens)
        blocks = torch.tensor(table[:-(-n // BS)], dtype=torch.long).cuda()
        for i in range(LAYERS):
            k, v = _kv(tokens, list(range(n)), i)
            for cache, want in ((self.k[i], k), (self.v[i], v)):
                assert torch.equal(cache[blocks].flatten(0, 1)[:n].cpu(), want)

    def cached_is_right(self, tokens):
        """Whatever the prefix cache finds of a prompt holds the prompt's K/V."""
        free = self.alloc.num_free
        table, hits = self.alloc.new_seq_cached(tokens)
        self.holds(table, tokens[:hits * BS])
        self.alloc.free(table)
        assert self.alloc.num_free == free
        return hits


def _step(s, tables, tokens, nodes, g):
    """One step over all sequences; the accepted tokens join `tokens`."""
    B = len(tables)
    bases = [len(t) for t in tokens]
    parents = [tu.random_parents(n, g) for n in nodes]
    draft = [torch.randint(0, 3, (n,), generator=g) for n in nodes]
    target = [torch.randint(0, 3, (n,), generator=g) for n in nodes]
    for b in range(B):
        s.grow(tables[b], bases[b], bases[b] + nodes[b])
        depth = tu.ancestors(parents[b])[1]
        s.write(tables[b], [bases[b] + i for i in range(nodes[b])], draft[b].tolist(), [bases[b] + int(x) for x in depth])
    full = s.alloc.num_free
    mb = max(len(t) for t in tables)
    table = torch.tensor([t + [-1] * (mb - len(t)) for t in tables], dtype=torch.int32).cuda()
    start, width = tu.starts(nodes).cuda(), max(nodes)
    path, count, _ = pkv.draft_tree_accept(torch.cat(draft).cuda(), torch.cat(target).cuda(), torch.cat(parents).cuda(),
                                           start, width)
    pkv.kv_cache_compact(s.k, s.v, table, torch.tensor(bases, dtype=torch.int32).cuda(), path, count)
    released = 0
    for b in range(B):
        want, _ = tu.accept(parents[b], draft[b], target[b])
        assert path[b, :int(count[b])].tolist() == want
        tokens[b] += [int(draft[b][i]) for i in want]
        released += -(-(bases[b] + nodes[b]) // BS) - -(-len(tokens[b]) // BS)
        s.alloc.truncate(tables[b], len(tokens[b]))
        assert len(tables[b]) == -(-len(tokens[b]) // BS)
    assert s.alloc.num_free == full + released              # drafts' blocks are nobody else's
    for b in range(B):
        s.holds(tables[b], tokens[b])
        s.register(tables[b], tokens[b])


def test_steps_with_prefix_caching_and_rollback():
    g = torch.Generator().manual_seed(77)
    pkv.device_flags(clear=True)
    s = _Server()
    tokens = [[int(x) for x in torch.randint(0, 50, (n,), generator=g)] for n in (64, 5, 33)]
    tables = [s.start(t) for t in tokens]
    for _ in range(4):
        _step(s, tables, tokens, [20, 12, 17], g)
    assert all(s.cached_is_right(t) == len(t) // BS for t in tokens)
    # roll two sequences back into a registered block (one of them within its last block) and go on otherwise
    before = [list(t) for t in tokens]
    for b, left in ((0, 50), (2, len(tokens[2]) // BS * BS - 3)):
        s.alloc.truncate(tables[b], left)
        tokens[b] = tokens[b][:left]
        s.cached_is_right(before[b])
    for _ in range(3):
        _step(s, tables, tokens, [9, 12, 30], g)
        for t in tokens + before:
            s.cached_is_right(t)
    # a fork that is rolled back copies the block that it writes; the other keeps its tokens
    fork, forked = s.alloc.fork(tables[0]), list(tokens[0])
    left = len(forked) // BS * BS - 5
    s.alloc.truncate(fork, left)
    mine, other = [forked[:left]], [fork]
    _step(s, other, mine, [14], g)
    s.holds(tables[0], tokens[0])
    s.holds(fork, mine[0])
    for t in tokens + before + mine:
        s.cached_is_right(t)
    # positions dropped from the middle of a context: its rewritten blocks leave the prefix cache first
    n = len(tokens[0])
    keep = [i for i in range(8, n) if i % 3]
    s.alloc.free(fork)
    s.alloc.cache_remove(tables[0])
    old = list(tokens[0])
    pkv.kv_cache_compact(s.k, s.v, torch.tensor([tables[0]], dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda(),
                         torch.tensor([list(range(8)) + keep], dtype=torch.int32).cuda(),
                         torch.tensor([8 + len(keep)], dtype=torch.int32).cuda())
    s.alloc.truncate(tables[0], 8 + len(keep))
    for t in tokens[1:] + before + mine + [old]:
        s.cached_is_right(t)
    for t in tables:
        s.alloc.free(t)
    assert s.alloc.num_free == POOL and pkv.device_flags() == 0
