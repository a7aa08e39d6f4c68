"""Compaction of kept cells on the GPU, bit for bit against index arithmetic."""
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from paged_kv_cache_468_b200 import pagedkv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_flags():
    pkv.device_flags(clear=True)
    yield
    assert pkv.device_flags() == 0


def _case(spans, kept, starts, layers=1, Hkv=2, D=64, bs=16, dtype=torch.bfloat16, seed=0):
    """spans[b]: tokens behind start; kept[b]: a count, or the positions themselves."""
    g = torch.Generator().manual_seed(seed)
    B = len(spans)
    pages = [max(1, -(-(a + s) // bs)) for a, s in zip(starts, spans)]
    NB = sum(pages) + 3
    order = torch.randperm(NB, generator=g).to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    lists = [torch.randperm(s, generator=g)[:k].sort().values.tolist() if isinstance(k, int) else list(k)
             for s, k in zip(spans, kept)]
    K = max(1, max(len(x) for x in lists))
    keep = torch.tensor([x + [-5] * (K - len(x)) for x in lists], dtype=torch.int32)
    caches = [torch.randint(-32768, 32768, (NB, bs, Hkv, D), generator=g, dtype=torch.int16).view(dtype)
              for _ in range(2 * layers)]
    return dict(caches=caches, layers=layers, table=table, starts=torch.tensor(starts, dtype=torch.int32), keep=keep,
                lens=torch.tensor([len(x) for x in lists], dtype=torch.int32), lists=lists, bs=bs)


def _expect(c):
    out = []
    for cache in c["caches"]:
        before, after = cache.view(torch.int16), cache.view(torch.int16).clone()
        for b, kept in enumerate(c["lists"]):
            for i, k in enumerate(kept):
                s, d = int(c["starts"][b]) + k, int(c["starts"][b]) + i
                after[int(c["table"][b, d // c["bs"]]), d % c["bs"]] = before[int(c["table"][b, s // c["bs"]]), s % c["bs"]]
        out.append(after)
    return out


def _run(c, **kw):
    d = [x.cuda() for x in c["caches"]]
    n = c["layers"]
    pkv.kv_cache_compact(d[:n], d[n:], c["table"].cuda(), c["starts"].cuda(), c["keep"].cuda(), c["lens"].cuda(), **kw)
    return d


def _check(c, got):
    for x, want in zip(got, _expect(c)):
        assert torch.equal(x.view(torch.int16).cpu(), want)


@pytest.mark.parametrize("Hkv,D,bs", [(1, 8, 16), (2, 64, 16), (8, 128, 32), (5, 40, 5), (3, 24, 7)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_small(Hkv, D, bs, dtype):
    c = _case([20, 1, 40, 9], [5, 1, [0, 1, 2, 30, 39], 0], [33, 0, 7, 11], 3, Hkv, D, bs, dtype, seed=D)
    _check(c, _run(c))


@pytest.mark.parametrize("share", [0.02, 0.5, 0.97, 1.0])
def test_long_lists(share):
    spans = [3000, 1, 517, 2048]
    c = _case(spans, [max(1, int(s * share)) for s in spans], [0, 5, 100, 31], 2, 2, 64, 16, seed=int(share * 100))
    _check(c, _run(c))


def test_patterns_that_overlap_most():
    # one token dropped at the front (every cell moves by one), the last ones kept, alternating, nothing moves
    n = 2500
    c = _case([n] * 5, [range(1, n), range(n - 100, n), range(0, n, 2), range(n), [n - 1]], [0, 1, 15, 16, 17], 1, 2, 32, 16, seed=9)
    _check(c, _run(c))


def test_many_layers_and_one_tensor_per_cache():
    c = _case([30, 12], [7, 12], [9, 0], 130, 1, 16, 16, seed=2)        # more layers than one launch takes
    _check(c, _run(c))
    c = _case([30, 12], [7, 5], [9, 0], 1, seed=3)
    d = [x.cuda() for x in c["caches"]]
    pkv.kv_cache_compact(d[0], d[1], c["table"].cuda(), c["starts"].cuda(), c["keep"].cuda(), c["lens"].cuda())
    _check(c, d)


def test_nothing_to_do():
    c = _case([30, 12], [[], []], [9, 0], 1, seed=4)
    _check(c, _run(c))
    c["keep"] = torch.zeros(2, 0, dtype=torch.int32)
    _check(c, _run(c))


def test_bad_entries_are_flagged_and_other_sequences_unharmed():
    c = _case([30, 200, 40], [7, [3, 2, 90, 10000, 150], 9], [9, 0, 3], 1, seed=5)
    got = _run(c)
    assert pkv.device_flags() == pagedkv.DEVFLAG_INDEX_RANGE
    mine = set(c["table"][1].tolist())
    c["lists"][1] = []
    for x, want in zip(got, _expect(c)):
        rest = [p for p in range(x.shape[0]) if p not in mine]
        assert torch.equal(x.view(torch.int16).cpu()[rest], want[rest])
    for key, b, value in (("starts", 0, -1), ("starts", 2, 10 ** 6), ("lens", 2, -1), ("lens", 2, 10 ** 6)):
        c = _case([30, 200, 40], [7, 50, 9], [9, 0, 3], 1, seed=6)
        c[key] = c[key].clone()
        c[key][b] = value
        got = _run(c)
        assert pkv.device_flags() == pagedkv.DEVFLAG_CONTEXT_RANGE
        c["lists"][b] = []                                   # the sequence is skipped
        c[key][b] = 0
        _check(c, got)
    c = _case([30, 200], [7, 50], [9, 0], 1, seed=7)
    c["table"][1, 1] = 10 ** 6
    _run(c)
    assert pkv.device_flags() == pagedkv.DEVFLAG_BLOCK_RANGE


def test_repeats_in_a_graph_on_a_stream_and_with_a_workspace():
    c = _case([3000, 40], [1500, 9], [0, 3], 2, 2, 64, 16, seed=8)
    want = _expect(c)
    start = [x.cuda() for x in c["caches"]]
    d = [x.clone() for x in start]
    args = (d[:2], d[2:], c["table"].cuda(), c["starts"].cuda(), c["keep"].cuda(), c["lens"].cuda())
    need = pkv.compact_workspace_bytes(2, 2, c["keep"].shape[1], 2, 64)
    ws = torch.full((max(1, need),), 255, dtype=torch.uint8).cuda()      # whatever it held before
    side = torch.cuda.Stream()

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(x.view(torch.int16).cpu(), w) for x, w in zip(d, want))

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_cache_compact(*args, workspace=ws)
    for way in (lambda: graph.replay(), lambda: graph.replay(), lambda: pkv.kv_cache_compact(*args, workspace=ws),
                lambda: pkv.kv_cache_compact(*args, stream=side)):
        for x, y in zip(d, start):
            x.copy_(y)
        torch.cuda.synchronize()
        way()
        assert same()


def test_large_batch_and_two_graphs_with_one_workspace():
    g = torch.Generator().manual_seed(12)
    spans = [int(x) for x in torch.randint(0, 300, (900,), generator=g)]
    kept = [int(torch.randint(0, s + 1, (1,), generator=g)) for s in spans]
    starts = [int(x) for x in torch.randint(0, 40, (900,), generator=g)]
    cases = [_case(spans, kept, starts, 1, 1, 32, 16, seed=13), _case([2000, 700], [900, 699], [3, 0], 2, 2, 64, 16, seed=14)]
    need = max(pkv.compact_workspace_bytes(c["layers"], len(c["lists"]), c["keep"].shape[1], c["caches"][0].shape[2],
                                           c["caches"][0].shape[3]) for c in cases)
    ws = torch.full((need,), 255, dtype=torch.uint8).cuda()
    graphs, held = [], []
    for c in cases:
        d = [x.cuda() for x in c["caches"]]
        n = c["layers"]
        args = (d[:n], d[n:], c["table"].cuda(), c["starts"].cuda(), c["keep"].cuda(), c["lens"].cuda())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pkv.kv_cache_compact(*args, workspace=ws)
        held.append((d, args))
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for c, (d, _) in zip(cases, held):
        _check(c, d)


@pytest.mark.parametrize("K", [16, 17, 256, 257])
def test_list_lengths_where_the_kernel_changes(K):
    c = _case([3 * K, K, K + 1], [K, K, K], [0, 20, 7], 2, 3, 40, 16, seed=K)
    _check(c, _run(c))
