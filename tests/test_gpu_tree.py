"""Drafted token trees on the GPU: ancestor bits, attention over the paged
cache and greedy acceptance against 64-bit references, and a whole step."""
import numpy as np
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from paged_kv_cache_468_b200 import pagedkv
from tests import tree_util as tu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_flags():
    pkv.device_flags(clear=True)
    yield
    assert pkv.device_flags() == 0


def _cuda(c):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}


def _attend(d, **kw):
    return pkv.paged_attention_tree(d["query"], d["query_start"], d["max_query_len"], d["tree_mask"],
                                    d["key_cache"], d["value_cache"], d["block_tables"], d["context_lens"],
                                    d["scale"], **kw)


def _check(c, out):
    ref, tol = tu.attend_reference(c)
    err = (out.double().cpu() - ref).abs()
    assert torch.isfinite(out).all()
    over = err - tol
    assert (over <= 0).all(), (float(err.max()), float(over.max()), np.unravel_index(int(over.argmax()), over.shape))


# ---- ancestor bits ----
@pytest.mark.parametrize("nodes", [[1], [32], [33, 0, 1, 31], [64, 65, 5], [0, 0, 7], [1000, 1024, 257]])
@pytest.mark.parametrize("chain", [False, True])
def test_mask_and_positions(nodes, chain):
    g = torch.Generator().manual_seed(sum(nodes))
    parents = [tu.random_parents(n, g, chain) for n in nodes]
    lens = torch.tensor([n + 3 * b for b, n in enumerate(nodes)], dtype=torch.int32)
    width = max(nodes)
    mask, pos = pkv.draft_tree_mask(torch.cat(parents).cuda(), tu.starts(nodes).cuda(), width, lens.cuda())
    at = 0
    for b, n in enumerate(nodes):
        bits, depth = tu.ancestors(parents[b])
        assert torch.equal(mask[at:at + n].cpu(), tu.pack(bits, -(-width // 32)))
        assert torch.equal(pos[at:at + n].cpu().long(), torch.from_numpy(depth + 3 * b))
        at += n


def test_mask_forest_wider_rows_and_rows_behind():
    # several roots; rows wider than any tree; rows behind the last sequence stay
    parents = torch.tensor([-1, -1, 0, 1, -1, 3, 7, 7], dtype=torch.int32)
    start = torch.tensor([0, 6], dtype=torch.int32)
    mask, pos = pkv.draft_tree_mask(parents.cuda(), start.cuda(), 70, torch.tensor([6], dtype=torch.int32).cuda())
    bits, depth = tu.ancestors(parents[:6])
    assert mask.shape == (8, 3)
    assert torch.equal(mask[:6].cpu(), tu.pack(bits, 3))
    assert torch.equal(pos[:6].cpu().long(), torch.from_numpy(depth))


def test_mask_bad_parents_and_bad_sequences_are_flagged():
    parents = torch.tensor([-1, 1, 5, -2, 2], dtype=torch.int32).cuda()     # 1, 2, 3: not earlier nodes
    start = torch.tensor([0, 5], dtype=torch.int32).cuda()
    mask, pos = pkv.draft_tree_mask(parents, start, 5, torch.tensor([9], dtype=torch.int32).cuda())
    assert mask[:, 0].tolist() == [1, 2, 4, 8, 16 + 4]
    assert pos.tolist() == [4, 4, 4, 4, 5]
    assert pkv.device_flags() == pagedkv.DEVFLAG_INDEX_RANGE
    for s, lens, width in (([0, 6], [9], 5), ([0, 5], [4], 5), ([3, 1], [9], 5), ([-1, 2], [9], 5), ([0, 5], [9], 4)):
        pkv.draft_tree_mask(parents, torch.tensor(s, dtype=torch.int32).cuda(), width,
                            torch.tensor(lens, dtype=torch.int32).cuda())
        assert pkv.device_flags() == pagedkv.DEVFLAG_CONTEXT_RANGE, s


# ---- acceptance ----
@pytest.mark.parametrize("nodes", [[1], [32], [33, 0, 2, 31], [1024, 300]])
@pytest.mark.parametrize("vocab", [2, 1000])
def test_accept(nodes, vocab):
    g = torch.Generator().manual_seed(vocab + sum(nodes))
    parents = [tu.random_parents(n, g) for n in nodes]
    draft = [torch.randint(0, vocab, (n,), generator=g) for n in nodes]
    target = [torch.randint(0, vocab, (n,), generator=g) for n in nodes]
    for p, d, t in zip(parents, draft, target):           # a long accepted path
        here = 0
        while len(p) and torch.rand(1, generator=g) < 0.95:
            below = [c for c in range(len(p)) if int(p[c]) == here]
            if not below:
                break
            t[here] = d[below[-1]]
            here = below[-1]
    path, lens, following = pkv.draft_tree_accept(torch.cat(draft).cuda(), torch.cat(target).cuda(),
                                                  torch.cat(parents).cuda(), tu.starts(nodes).cuda(), max(nodes))
    for b, n in enumerate(nodes):
        want, token = tu.accept(parents[b], draft[b], target[b])
        assert path[b].tolist() == want + [-1] * (max(nodes) - len(want))
        assert int(lens[b]) == len(want) and int(following[b]) == token


def test_accept_chain_of_all_nodes_and_bad_sequences():
    n = 1024
    tokens = torch.arange(n) + (1 << 40)                   # tokens past 32 bits
    path, lens, following = pkv.draft_tree_accept(tokens.cuda(), (tokens + 1).cuda(),
                                                  tu.random_parents(n, None, chain=True).cuda(),
                                                  tu.starts([n]).cuda(), n)
    assert path[0].tolist() == list(range(n)) and int(lens[0]) == n and int(following[0]) == (1 << 40) + n
    start = torch.tensor([0, n + 1], dtype=torch.int32).cuda()
    path, lens, following = pkv.draft_tree_accept(tokens.cuda(), tokens.cuda(), torch.zeros(n, dtype=torch.int32).cuda() - 1,
                                                  start, n)
    assert int(lens[0]) == 0 and int(following[0]) == -1 and (path == -1).all()
    assert pkv.device_flags() == pagedkv.DEVFLAG_CONTEXT_RANGE
    parents = torch.tensor([-1, 0, 2], dtype=torch.int32).cuda()   # node 2 below itself
    same = torch.zeros(3, dtype=torch.int64).cuda()
    path, lens, _ = pkv.draft_tree_accept(same, same, parents, tu.starts([3]).cuda(), 3)
    assert path[0].tolist() == [0, 1, -1]
    assert pkv.device_flags() == pagedkv.DEVFLAG_INDEX_RANGE


# ---- attention ----
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_ragged(D, bs, dtype):
    c = tu.tree_case([5, 0, 1, 33, 17, 2], [40, 100, 0, 63, 300, 1], 8, 2, D, bs, dtype, seed=D + bs)
    _check(c, _attend(_cuda(c)))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (10, 2), (6, 1), (14, 2), (8, 1), (5, 5)])
def test_attend_group_sizes(Hq, Hkv):
    c = tu.tree_case([19, 7, 45], [77, 0, 130], Hq, Hkv, 64, 16, "bf16", seed=Hq)
    _check(c, _attend(_cuda(c)))


@pytest.mark.parametrize("n,base", [(1, 0), (1, 1), (1, 63), (1, 64), (2, 62), (64, 0), (65, 0), (16, 48), (16, 49),
                                    (128, 0), (129, 31), (31, 33), (33, 191)])
@pytest.mark.parametrize("bs", [16, 32])
def test_attend_borders(n, base, bs):
    # pages and key tiles that end inside, before and behind the tree
    c = tu.tree_case([n], [base], 4, 1, 128, bs, "f16", seed=n * 1000 + base)
    _check(c, _attend(_cuda(c)))


def test_attend_wide_tree_many_rows():
    # 300 nodes x 8 heads of one kv head: many row tiles
    c = tu.tree_case([300, 3, 150], [90, 700, 0], 8, 1, 64, 16, "bf16", seed=3)
    _check(c, _attend(_cuda(c)))


def test_attend_long_context():
    c = tu.tree_case([9, 30], [5000, 2111], 4, 1, 128, 32, "bf16", seed=4)
    _check(c, _attend(_cuda(c)))


def test_attend_any_bits_empty_rows_and_bits_past_the_tree():
    g = torch.Generator().manual_seed(5)
    nodes, bases = [40, 6, 70, 3], [0, 0, 100, 20]
    bits = []
    for n in nodes:
        x = (torch.rand(n, 96, generator=g) < 0.3).numpy()
        x[n // 2] = False                                  # no drafted key at all
        x[n // 2, n:] = True                               # bits of nodes that do not exist
        bits.append(x)
    c = tu.tree_case(nodes, bases, 4, 2, 64, 16, "bf16", seed=6, bits=bits, max_query_len=96)
    out = _attend(_cuda(c))
    _check(c, out)
    assert (out[20] == 0).all() and (out[43] == 0).all()   # rows that see nothing


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attend_large_and_growing_scores(dtype):
    c = tu.tree_case([12, 30], [500, 0], 8, 2, 128, 16, dtype, seed=7, q_scale=30.0)
    for k in c["keys"]:
        k *= (0.2 + torch.arange(k.shape[0]) / k.shape[0] * 3)[:, None, None].to(k.dtype)
    for b, k in enumerate(c["keys"]):
        for j in range(k.shape[0]):
            c["key_cache"][int(c["block_tables"][b, j // 16]), j % 16] = k[j]
    _check(c, _attend(_cuda(c)))


def test_attend_nonfinite_cells_that_a_row_does_not_see():
    # node 3 holds infinities and NaN in K and V: rows that do not see it stay finite, the others follow the formula
    parents = torch.tensor([-1, 0, 0, 1, 1, 3, 2], dtype=torch.int32)
    bits = tu.ancestors(parents)[0]
    for base in (0, 57, 200):
        c = tu.tree_case([7], [base], 4, 2, 64, 16, "bf16", seed=8, bits=[bits])
        page, cell = int(c["block_tables"][0, (base + 3) // 16]), (base + 3) % 16
        c["value_cache"][page, cell, :, 5] = float("inf")
        c["value_cache"][page, cell, :, 6] = float("nan")
        c["value_cache"][page, cell, :, 7] = float("-inf")
        out = _attend(_cuda(c)).cpu()
        blind = [0, 1, 2, 4, 6]
        c["values"][0][base + 3] = 0.0                     # (blind rows give it no weight)
        ref, tol = tu.attend_reference(c)
        assert ((out.double() - ref).abs() <= tol)[blind].all()
        for i in (3, 5):
            assert (out[i, :, 5] == float("inf")).all() and out[i, :, 6].isnan().all() and (out[i, :, 7] == float("-inf")).all()
            assert out[i, :, :5].isfinite().all() and out[i, :, 8:].isfinite().all()
        c["key_cache"][page, cell] = float("nan")          # a NaN score poisons the rows that see it alone
        out = _attend(_cuda(c)).cpu()
        assert ((out.double() - ref).abs() <= tol)[blind].all()
        assert out[[3, 5]].isnan().all()


def test_attend_rows_outside_sequences_stay():
    c = tu.tree_case([5, 9], [30, 8], 4, 2, 64, 16, "f16", seed=9)
    d = _cuda(c)
    q = torch.cat([d["query"], d["query"][:3]])
    out = torch.full_like(q, 7.0)
    d2 = dict(d, query=q, tree_mask=torch.cat([d["tree_mask"], d["tree_mask"][:3]]))
    got = _attend(d2, out=out)
    assert got is out and (out[14:] == 7.0).all()
    _check(c, out[:14])


def test_attend_contradicting_lengths_are_flagged_and_skipped():
    c = tu.tree_case([5, 9, 4], [30, 8, 12], 4, 2, 64, 16, "f16", seed=10)
    d = _cuda(c)
    want = _attend(d)
    for b, length in ((1, 8), (1, -3), (1, 10 ** 6), (0, 4)):
        lens = d["context_lens"].clone()
        lens[b] = length
        out = torch.full_like(want, 7.0)
        _attend(dict(d, context_lens=lens), out=out)
        assert pkv.device_flags() == pagedkv.DEVFLAG_CONTEXT_RANGE
        lo, hi = int(c["query_start"][b]), int(c["query_start"][b + 1])
        assert (out[lo:hi] == 7.0).all()
        rest = torch.ones(18, dtype=torch.bool)
        rest[lo:hi] = False
        assert torch.equal(out[rest.cuda()], want[rest.cuda()])


def test_attend_page_outside_the_pool_is_flagged():
    c = tu.tree_case([5], [50], 4, 2, 64, 16, "f16", seed=11)
    d = _cuda(c)
    d["block_tables"][0, 1] = 10 ** 6
    _attend(d)
    assert pkv.device_flags() == pagedkv.DEVFLAG_BLOCK_RANGE


def test_attend_agrees_with_decode_and_prefill():
    # a tree of one node is a decode step, a chain a causal chunk
    c = tu.tree_case([1, 1, 1], [200, 64, 0], 8, 2, 128, 16, "bf16", seed=12)
    d = _cuda(c)
    one = pkv.paged_attention_decode(d["query"], d["key_cache"], d["value_cache"], d["block_tables"],
                                     d["context_lens"], d["scale"])
    ref, tol = tu.attend_reference(c)
    assert ((one.double().cpu() - ref).abs() <= tol).all()
    _check(c, _attend(d))
    chain = [np.tril(np.ones((n, n), dtype=bool)) for n in (50, 9)]
    c = tu.tree_case([50, 9], [33, 400], 8, 2, 128, 16, "bf16", seed=13, bits=chain)
    d = _cuda(c)
    many = pkv.paged_attention_prefill(d["query"], d["query_start"], 50, d["key_cache"], d["value_cache"],
                                       d["block_tables"], d["context_lens"], d["scale"])
    _check(c, many)
    _check(c, _attend(d))


def test_attend_repeats_bit_for_bit_and_in_a_graph_and_on_a_stream():
    c = tu.tree_case([16] * 24, list(range(10, 1210, 50)), 8, 2, 128, 16, "bf16", seed=14)
    d = _cuda(c)
    first = _attend(d)
    for _ in range(20):
        assert torch.equal(_attend(d), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _attend(d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _attend(d)
    # other lengths and masks in the same buffers, then back: a replay follows the buffers
    lens = d["context_lens"].clone()
    d["context_lens"].sub_(3)
    want = _attend(d)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want)
    d["context_lens"].copy_(lens)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, first)


# A wide table makes the library plan for long contexts: equal shares of key
# tiles per CTA (over 16 rows), parts of a context (up to 16), instead of
# clusters.  The same contexts then run through the other kernels.
_WIDE = {16: 4096, 32: 2048}


@pytest.mark.parametrize("Hq,Hkv,nodes", [(8, 2, [5, 0, 1, 33, 17, 2]), (3, 1, [50, 1, 90]), (8, 1, [300, 3, 150]),
                                          (4, 2, [2, 8, 1, 0, 5]), (1, 1, [16, 3, 9]), (7, 1, [2, 1])])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32), (128, 16), (64, 32)])
def test_attend_planned_for_long_contexts(Hq, Hkv, nodes, D, bs):
    bases = [40, 100, 0, 63, 1300, 1][:len(nodes)]
    c = tu.tree_case(nodes, bases, Hq, Hkv, D, bs, "bf16" if D == 64 else "f16", seed=D + bs + Hq, columns=_WIDE[bs])
    d = _cuda(c)
    out = _attend(d)
    _check(c, out)
    for _ in range(5):
        assert torch.equal(_attend(d), out)


@pytest.mark.parametrize("n,base", [(1, 0), (1, 63), (20, 0), (33, 31), (16, 48), (16, 49), (65, 0), (129, 31), (31, 33)])
def test_attend_borders_planned_for_long_contexts(n, base):
    c = tu.tree_case([n], [base], 4, 1, 128, 16, "f16", seed=n * 1000 + base, columns=_WIDE[16])
    _check(c, _attend(_cuda(c)))


def test_attend_any_bits_planned_for_long_contexts():
    g = torch.Generator().manual_seed(25)
    nodes, bases = [40, 6, 70, 3], [0, 0, 100, 20]
    bits = [(torch.rand(n, 96, generator=g) < 0.3).numpy() for n in nodes]
    for x, n in zip(bits, nodes):
        x[n // 2] = False
        x[n // 2, n:] = True
    c = tu.tree_case(nodes, bases, 4, 2, 64, 16, "bf16", seed=26, bits=bits, max_query_len=96, columns=_WIDE[16])
    out = _attend(_cuda(c))
    _check(c, out)
    assert (out[20] == 0).all() and (out[43] == 0).all()


@pytest.mark.parametrize("heads", [(4, 2), (16, 2)])
@pytest.mark.parametrize("columns", [0, 4096])
def test_attend_nonfinite_cells_in_every_kernel(heads, columns):
    parents = torch.tensor([-1, 0, 0, 1, 1, 3, 2], dtype=torch.int32)
    bits = tu.ancestors(parents)[0]
    nodes, bases = [7, 7, 7], [200, 0, 57]
    c = tu.tree_case(nodes, bases, *heads, 128, 16, "f16", seed=28, bits=[bits] * 3, columns=columns)
    for b, base in enumerate(bases):
        page, cell = int(c["block_tables"][b, (base + 3) // 16]), (base + 3) % 16
        c["value_cache"][page, cell, :, 70] = float("inf")
        c["value_cache"][page, cell, :, 6] = float("nan")
        c["key_cache"][page, cell, :, 9] = float("nan") if b == 2 else c["key_cache"][page, cell, :, 9]
        c["values"][b][base + 3] = 0.0
    out = _attend(_cuda(c)).cpu()
    ref, tol = tu.attend_reference(c)
    blind = [7 * b + i for b in range(3) for i in (0, 1, 2, 4, 6)]
    assert ((out.double() - ref).abs() <= tol)[blind].all()
    for b in range(3):
        for i in (3, 5):
            row = out[7 * b + i]
            if b == 2:
                assert row.isnan().all()                   # a NaN score
            else:
                assert (row[:, 70] == float("inf")).all() and row[:, 6].isnan().all()
                assert row[:, :6].isfinite().all() and row[:, 7:70].isfinite().all() and row[:, 71:].isfinite().all()


# 17 to 64 query rows per item and head_dim 128 over a wide table: the kernel
# with keys as the rows of its products.
@pytest.mark.parametrize("Hq,Hkv,nodes", [(8, 2, [16, 3, 0, 9, 1]), (1, 1, [64, 33, 1, 17, 2]), (5, 1, [12, 1, 5, 0, 7]),
                                          (6, 2, [21, 7, 10, 1, 0]), (8, 1, [5, 8, 1, 3, 4]), (4, 1, [8, 5, 7, 1, 2])])
@pytest.mark.parametrize("dtype,bs", [("f16", 16), ("bf16", 32)])
def test_attend_up_to_64_rows_planned_for_long_contexts(Hq, Hkv, nodes, dtype, bs):
    for k, bases in enumerate(([127, 1300, 9, 0, 128], [0, 64, 50, 3001, 119], [63, 0, 700, 255, 1])):
        c = tu.tree_case(nodes, bases, Hq, Hkv, 128, bs, dtype, seed=50 + k, columns=_WIDE[bs])
        d = _cuda(c)
        out = _attend(d)
        _check(c, out)
        for _ in range(3):
            assert torch.equal(_attend(d), out)


@pytest.mark.parametrize("n,base", [(9, 0), (16, 0), (16, 111), (16, 112), (16, 113), (15, 113), (13, 300), (16, 240), (10, 64)])
@pytest.mark.parametrize("bs", [16, 32])
def test_attend_borders_up_to_64_rows(n, base, bs):
    c = tu.tree_case([n], [base], 4, 1, 128, bs, "bf16", seed=n * 1000 + base, columns=_WIDE[bs])
    _check(c, _attend(_cuda(c)))


def test_attend_any_bits_up_to_64_rows():
    g = torch.Generator().manual_seed(51)
    nodes, bases = [40, 6, 64, 3], [0, 0, 100, 20]
    bits = [(torch.rand(n, 64, generator=g) < 0.3).numpy() for n in nodes]
    for x, n in zip(bits, nodes):
        x[n // 2] = False
        x[n // 2, n:] = True
    c = tu.tree_case(nodes, bases, 2, 2, 128, 16, "f16", seed=52, bits=bits, max_query_len=64, columns=_WIDE[16])
    out = _attend(_cuda(c))
    _check(c, out)
    assert (out[20] == 0).all() and (out[43] == 0).all()


@pytest.mark.parametrize("columns", [0, 4096])
@pytest.mark.parametrize("nodes", [[4, 3], [12, 16], [12, 30]])
def test_attend_moving_maxima_in_every_kernel(columns, nodes):
    # scores that grow along the keys, that fall, and one early key far above or below the others
    for shape in ("grow", "fall", "high", "low"):
        c = tu.tree_case(nodes, [500, 700], 8, 2, 128, 16, "bf16", seed=53, q_scale=30.0, columns=columns)
        for k in c["keys"]:
            n = k.shape[0]
            f = torch.arange(n) / n * 3 + 0.2
            if shape == "fall":
                f = f.flip(0)
            if shape in ("high", "low"):
                f = torch.full((n,), 0.05)
                f[0 if shape == "low" else 150] = 4.0
            k *= f[:, None, None].to(k.dtype)
        for b, k in enumerate(c["keys"]):
            for j in range(k.shape[0]):
                c["key_cache"][int(c["block_tables"][b, j // 16]), j % 16] = k[j]
        _check(c, _attend(_cuda(c)))


@pytest.mark.parametrize("heads", [(4, 2), (16, 2)])
@pytest.mark.parametrize("columns", [0, 4096])
@pytest.mark.parametrize("nodes", [[2, 1], [7, 4], [25, 13]])
def test_attend_nan_query_row_stays_its_own(heads, columns, nodes):
    c = tu.tree_case(nodes, [300, 20], *heads, 128, 16, "f16", seed=54, columns=columns)
    d = _cuda(c)
    d["query"][1, 1, 17] = float("nan")
    out = _attend(d)
    assert out[1, 1].isnan().all()
    ref, tol = tu.attend_reference(c)
    fine = torch.ones(sum(nodes), heads[0], dtype=torch.bool)
    fine[1, 1] = False
    assert ((out.double().cpu() - ref).abs() <= tol)[fine].all()


def test_attend_negative_zero_and_tiny_scale_up_to_64_rows():
    for scale in (-0.3, 0.0, 1e-6):
        c = tu.tree_case([20, 5], [300, 0], 4, 2, 128, 16, "bf16", seed=55, columns=_WIDE[16])
        c["scale"] = scale
        _check(c, _attend(_cuda(c)))


def test_attend_many_short_sequences():
    # more sequences than a CTA has threads, some without rows; shares hold many small items
    g = torch.Generator().manual_seed(27)
    nodes = [int(x) for x in torch.randint(0, 9, (700,), generator=g)]
    bases = [int(x) for x in torch.randint(0, 40, (700,), generator=g)]
    for heads, columns in (((4, 1), 0), ((4, 1), 600), ((1, 1), 0)):
        c = tu.tree_case(nodes, bases, *heads, 64, 16, "bf16", seed=29, columns=columns)
        _check(c, _attend(_cuda(c)))


def test_attend_largest_tree():
    c = tu.tree_case([1024, 700], [17, 64], 2, 1, 64, 16, "bf16", seed=30)
    _check(c, _attend(_cuda(c)))
    c = tu.tree_case([1024], [30], 1, 1, 128, 32, "f16", seed=31, columns=4096)
    _check(c, _attend(_cuda(c)))


def test_attend_negative_zero_and_tiny_scale():
    for scale in (-0.3, 0.0, 1e-6):
        c = tu.tree_case([20, 5], [90, 0], 4, 2, 64, 16, "bf16", seed=32)
        c["scale"] = scale
        _check(c, _attend(_cuda(c)))
        c = tu.tree_case([3, 5], [90, 0], 2, 2, 64, 16, "bf16", seed=33)
        c["scale"] = scale
        _check(c, _attend(_cuda(c)))


def test_two_graphs_share_a_workspace_and_two_streams_have_their_own():
    cases = [tu.tree_case([30] * 6, [100 * i for i in range(6)], 4, 2, 64, 16, "bf16", seed=40 + k, columns=4096) for k in range(2)]
    ds = [_cuda(c) for c in cases]
    need = pkv.tree_workspace_bytes(6, 30, 180, 4, 2, 64, 4096, 16)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8).cuda()
    want = [_attend(d) for d in ds]
    graphs, held = [], []
    for d in ds:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(_attend(d, workspace=ws))
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got = [[_attend(d, stream=s) for d, s in zip(ds, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for outs in got for a, b in zip(outs, want))


# ---- a whole step ----
def test_verification_step_end_to_end():
    """Draft, write, mask, attend, accept, compact, truncate; then a decode over what is left equals
    one over a cache that only ever held the accepted tokens."""
    Hq, Hkv, D, bs, layers = 8, 2, 64, 16, 3
    g = torch.Generator().manual_seed(15)
    bases, nodes = [33, 5, 64], [20, 12, 17]
    alloc = pkv.BlockAllocator(64, bs, shuffle_seed=3)
    tables = [alloc.new_seq(n) for n in bases]
    kcs = [torch.zeros(64, bs, Hkv, D, dtype=torch.bfloat16).cuda() for _ in range(layers)]
    vcs = [torch.zeros(64, bs, Hkv, D, dtype=torch.bfloat16).cuda() for _ in range(layers)]
    for b, n in enumerate(nodes):
        alloc.append(tables[b], bases[b], bases[b] + n)
    free_before = alloc.num_free
    mb = max(len(t) for t in tables)
    bt = torch.tensor([t + [-1] * (mb - len(t)) for t in tables], dtype=torch.int32).cuda()
    kv = {}
    for b in range(3):
        L = bases[b] + nodes[b]
        slots = torch.tensor([tables[b][p // bs] * bs + p % bs for p in range(L)]).cuda()
        for i in range(layers):
            k, v = (torch.randn(L, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
            pkv.kv_cache_write(k, v, slots, kcs[i], vcs[i])
            kv[b, i] = k, v
    parents = [tu.random_parents(n, g) for n in nodes]
    draft = [torch.randint(0, 3, (n,), generator=g) for n in nodes]
    target = [torch.randint(0, 3, (n,), generator=g) for n in nodes]
    start, width = tu.starts(nodes).cuda(), max(nodes)
    lens = torch.tensor([a + n for a, n in zip(bases, nodes)], dtype=torch.int32).cuda()
    mask, pos = pkv.draft_tree_mask(torch.cat(parents).cuda(), start, width, lens)
    q = torch.randn(sum(nodes), Hq, D, generator=g).to(torch.bfloat16).cuda()
    for i in range(layers):
        out = pkv.paged_attention_tree(q, start, width, mask, kcs[i], vcs[i], bt, lens, D ** -0.5)
        c = dict(query=q.cpu(), key_cache=kcs[i], dtype="bf16", nodes=nodes, bases=bases, scale=D ** -0.5,
                 bits=[tu.ancestors(p)[0] for p in parents], keys=[kv[b, i][0].cpu() for b in range(3)],
                 values=[kv[b, i][1].cpu() for b in range(3)])
        _check(c, out)
    path, count, following = pkv.draft_tree_accept(torch.cat(draft).cuda(), torch.cat(target).cuda(),
                                                   torch.cat(parents).cuda(), start, width)
    base = torch.tensor(bases, dtype=torch.int32).cuda()
    pkv.kv_cache_compact(kcs, vcs, bt, base, path, count)
    left = base + count
    for b in range(3):
        want, token = tu.accept(parents[b], draft[b], target[b])
        assert path[b, :len(want)].tolist() == want and int(following[b]) == token
        alloc.truncate(tables[b], int(left[b]))
        assert len(tables[b]) == -(-int(left[b]) // bs)
    assert alloc.num_free >= free_before
    bt = torch.tensor([t + [-1] * (mb - len(t)) for t in tables], dtype=torch.int32).cuda()
    q1 = torch.randn(3, Hq, D, generator=g).to(torch.bfloat16).cuda()
    for i in range(layers):
        got = pkv.paged_attention_decode(q1, kcs[i], vcs[i], bt, left, D ** -0.5)
        kc, vc = torch.zeros_like(kcs[0]), torch.zeros_like(vcs[0])
        for b in range(3):
            kept = list(range(bases[b])) + [bases[b] + j for j in path[b, :int(count[b])].tolist()]
            slots = torch.tensor([tables[b][p // bs] * bs + p % bs for p in range(len(kept))]).cuda()
            pkv.kv_cache_write(kv[b, i][0][kept].contiguous(), kv[b, i][1][kept].contiguous(), slots, kc, vc)
        assert torch.equal(got, pkv.paged_attention_decode(q1, kc, vc, bt, left, D ** -0.5))
