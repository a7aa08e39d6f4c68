"""The measured cases of the speculative-decoding operators over a paged KV cache.

A step of speculative decoding drafts a tree of tokens per sequence, writes
their K/V behind the sequence's committed tokens, lets every drafted token
attend over the committed tokens and its own ancestors, accepts the path that
the target model's answers confirm, and moves the accepted tokens' cells
together in the cache.  Its operators here:

  attend   paged_attention_tree   drafted tokens over the cache, masked by the tree
  mask     draft_tree_mask        parents -> packed ancestor bits and positions
  accept   draft_tree_accept      greedy verification: path, length, next token
  compact  kv_cache_compact       kept cells of each sequence moved together

`run` computes an operator in its plain form (elementary torch operations) or,
where `own` is true, through the framework's entry points.
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one interactive user, a small tree: the latency of a layer's call
        dict(name="attend one user", op="attend", batch=1, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16",
             len_lo=601, len_hi=601, nodes_lo=8, nodes_hi=8, idle=0),
        # a full serving batch at the headline's context lengths, a few nodes each
        dict(name="attend batch 256", op="attend", batch=256, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16",
             len_lo=512, len_hi=640, nodes_lo=6, nodes_hi=10, idle=0),
        # ragged lengths without grouped heads, odd tree sizes, some sequences not drafting
        dict(name="attend ragged mha", op="attend", batch=50, heads=40, kv_heads=40, dim=128, block=16, dtype="f16",
             len_lo=64, len_hi=2048, nodes_lo=1, nodes_hi=27, idle=7),
        # small heads, prompts shorter than the trees
        dict(name="attend tiny heads", op="attend", batch=33, heads=8, kv_heads=8, dim=64, block=16, dtype="f16",
             len_lo=1, len_hi=200, nodes_lo=1, nodes_hi=61, idle=0),
        # long contexts, wide trees: the largest call
        dict(name="attend long", op="attend", batch=8, heads=32, kv_heads=8, dim=128, block=32, dtype="bf16",
             len_lo=16384, len_hi=32768, nodes_lo=60, nodes_hi=64, idle=0),
        # trees of a serving batch, and of a batch with very wide trees
        dict(name="mask batch 64", op="mask", batch=64, nodes_lo=26, nodes_hi=33, len_lo=512, len_hi=640, idle=0),
        dict(name="mask wide", op="mask", batch=256, nodes_lo=500, nodes_hi=1000, len_lo=16, len_hi=2048, idle=5),
        dict(name="accept batch 64", op="accept", batch=64, nodes_lo=26, nodes_hi=33, idle=0),
        dict(name="accept wide", op="accept", batch=512, nodes_lo=300, nodes_hi=1000, idle=5),
        # accepted tokens of a step, all layers of a model in one call
        dict(name="compact accepted", op="compact", layers=16, batch=16, kv_heads=8, dim=128, block=16, dtype="bf16",
             len_lo=512, len_hi=640, span_lo=26, span_hi=33, keep=0.15, head=1),
        # tokens dropped from all over a context: the kept ones move together
        dict(name="compact ragged mha", op="compact", layers=1, batch=50, kv_heads=40, dim=128, block=16, dtype="f16",
             len_lo=0, len_hi=16, span_lo=64, span_hi=2031, keep=0.7, head=4),
        dict(name="compact long", op="compact", layers=1, batch=8, kv_heads=8, dim=128, block=32, dtype="bf16",
             len_lo=0, len_hi=0, span_lo=16384, span_hi=32768, keep=0.5, head=64),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    limit = {}
    for c in listed():
        w, size = work(c), _padded(c)
        top = limit.setdefault(c["op"], [0.0, 0.0, 0.0])
        limit[c["op"]] = [max(top[0], w["bytes"]), max(top[1], w["flops"]), max(top[2], size)]
    while True:
        c = _draw_once(rng)
        w = work(c)
        top = limit[c["op"]]
        if w["bytes"] <= top[0] and w["flops"] <= top[1] and _padded(c) <= top[2]:
            return c


def _draw_once(rng):
    op = rng.choice(["attend", "attend", "attend", "mask", "accept", "compact", "compact"])
    heads, kv_heads, dim, block = rng.choice(
        [(8, 8, 64, 16), (32, 8, 128, 16), (32, 8, 128, 32), (40, 40, 128, 16), (14, 2, 64, 16), (24, 8, 128, 32),
         (10, 2, 128, 16), (4, 4, 64, 32), (32, 4, 128, 16)])
    dtype = rng.choice(["f16", "bf16"])
    if op == "attend":
        hi, n = _log(rng, 1, 32768), _log(rng, 1, 256)
        return dict(op=op, batch=_log(rng, 1, 256), heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype,
                    len_lo=_log(rng, 1, hi), len_hi=hi, nodes_lo=_log(rng, 1, n), nodes_hi=n, idle=rng.choice([0, 0, 3, 7]))
    if op in ("mask", "accept"):
        n = _log(rng, 1, 1000)
        c = dict(op=op, batch=_log(rng, 1, 512), nodes_lo=_log(rng, 1, n), nodes_hi=n, idle=rng.choice([0, 0, 3, 7]))
        return dict(c, len_lo=rng.randint(0, 16), len_hi=rng.randint(16, 4096)) if op == "mask" else c
    hi = _log(rng, 1, 32768)
    return dict(op=op, layers=rng.choice([1, 2, 5, 16]), batch=_log(rng, 1, 64), kv_heads=kv_heads, dim=dim, block=block,
                dtype=dtype, len_lo=0, len_hi=rng.choice([0, 50, 1000]), span_lo=_log(rng, 1, hi), span_hi=hi,
                keep=round(rng.uniform(0.05, 0.95), 2), head=rng.choice([0, 1, 16]))


def _spread(lo, hi, n, step):
    """n whole numbers between lo and hi, in no order, that depend on the case alone."""
    return [lo + (i * step + step // 2) % (hi - lo + 1) for i in range(n)]


def _nodes(case):
    """Drafted tokens of each sequence; every idle-th sequence drafts none."""
    n = _spread(case["nodes_lo"], case["nodes_hi"], case["batch"], 7919)
    return [0 if case["idle"] and b % case["idle"] == case["idle"] - 1 else v for b, v in enumerate(n)]


def _lens(case):
    """Tokens of each sequence before the drafted ones (compact: before the first cell that may move)."""
    return _spread(case["len_lo"], case["len_hi"], case["batch"], 104729)


def _spans(case):
    """compact: tokens behind the start, and how many of them are kept."""
    spans = _spread(case["span_lo"], case["span_hi"], case["batch"], 7919)
    return spans, [max(1, int(s * case["keep"])) for s in spans]


def _padded(case):
    """Values of the largest padded array in the plain form."""
    if case["op"] == "attend":
        nodes, lens = _nodes(case), _lens(case)
        longest = max(a + b for a, b in zip(nodes, lens))
        return case["batch"] * max(case["heads"] * max(nodes) * longest, 2 * case["kv_heads"] * case["dim"] * longest)
    if case["op"] in ("mask", "accept"):
        return case["batch"] * max(1, max(_nodes(case))) ** 2
    return case["layers"] * 2 * case["kv_heads"] * case["dim"] * sum(a + b for a, b in zip(_lens(case), _spans(case)[0]))


def work(case):
    if case["op"] == "attend":
        nodes, lens = _nodes(case), _lens(case)
        row = case["dim"] * 2
        live = [(n, c + n) for n, c in zip(nodes, lens) if n > 0]
        width = -(-max(1, max(nodes)) // 32)
        size = sum(t for _, t in live) * case["kv_heads"] * row * 2       # K and V, each cell once
        size += sum(nodes) * (2 * case["heads"] * row + 4 * width)        # queries, outputs, mask rows
        size += sum(-(-t // case["block"]) * 4 for _, t in live) + 8 * case["batch"]
        pairs = sum(n * (t - n + 1) for n, t in live)                     # committed tokens and the node itself
        return {"bytes": size, "flops": 4 * case["dim"] * case["heads"] * pairs}
    if case["op"] == "mask":
        nodes = _nodes(case)
        width = -(-max(1, max(nodes)) // 32)
        return {"bytes": sum(nodes) * (4 + 4 * width + 4) + 8 * case["batch"], "flops": sum(nodes) * width}
    if case["op"] == "accept":
        nodes = _nodes(case)
        return {"bytes": sum(nodes) * (4 + 8 + 8) + case["batch"] * (4 * max(1, max(nodes)) + 4 + 8 + 4), "flops": sum(nodes)}
    spans, kept = _spans(case)
    # every kept token is read and written once, but for the leading ones that stay where they are
    moved = sum(max(0, k - min(case["head"], k)) for k in kept)
    cell = case["kv_heads"] * case["dim"] * 2 * 2 * case["layers"]
    return {"bytes": max(16, moved * cell * 2 + sum(kept) * 4), "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generators(seed):
    return torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed)


def _starts(counts):
    return torch.tensor([0] + counts).cumsum(0)


def _tree(nodes, host):
    """Parents of every node within its sequence: node 0 is the root, the others hang below a recent earlier node."""
    total = sum(nodes)
    index = torch.cat([torch.arange(n) for n in nodes]) if total else torch.zeros(0, dtype=torch.int64)
    back = 1 + (torch.rand(total, generator=host) ** 2 * 6).long()
    return torch.where(index > 0, (index - back).clamp(min=0), torch.tensor(-1)).to(torch.int32)


def _tables(totals, block, host):
    """A page table over a pool of pages in random order; entries behind a sequence's last page are -1."""
    pages = [-(-t // block) for t in totals]
    pool = max(1, sum(pages) + sum(pages) // 10)
    order = torch.randperm(pool, generator=host).to(torch.int32)
    table = torch.full((len(totals), max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = order[at:at + p]
        at += p
    return table, pool


def prepare(case, seed):
    host, dev = _generators(seed)
    s = {"op": case["op"]}
    if case["op"] == "attend":
        nodes, lens = _nodes(case), _lens(case)
        dt = _DT[case["dtype"]]
        totals = [n + c for n, c in zip(nodes, lens)]
        table, pool = _tables(totals, case["block"], host)
        shape = (pool, case["block"], case["kv_heads"], case["dim"])
        s["key_cache"] = torch.randn(shape, generator=dev, device="cuda", dtype=dt)
        s["value_cache"] = torch.randn(shape, generator=dev, device="cuda", dtype=dt)
        s["query"] = torch.randn((sum(nodes), case["heads"], case["dim"]), generator=dev, device="cuda", dtype=dt)
        s["block_tables"] = table.cuda()
        s["context_lens"] = torch.tensor(totals, dtype=torch.int32).cuda()
        s["query_start"] = _starts(nodes).to(torch.int32).cuda()
        s["max_query_len"] = max(1, max(nodes))
        s["scale"] = case["dim"] ** -0.5
        bits = _closure(_pad_parents(_tree(nodes, host).cuda(), s["query_start"], s["max_query_len"]))
        s["tree_mask"] = _unpad(_pack(bits), s["query_start"])
    elif case["op"] in ("mask", "accept"):
        nodes = _nodes(case)
        parents = _tree(nodes, host)
        start = _starts(nodes)
        s["parents"] = parents.cuda()
        s["query_start"] = start.to(torch.int32).cuda()
        s["max_query_len"] = max(1, max(nodes))
        if case["op"] == "mask":
            s["context_lens"] = torch.tensor([n + c for n, c in zip(nodes, _lens(case))], dtype=torch.int32).cuda()
        else:
            # tokens as a small vocabulary's argmax gives them; the target agrees with some child of most nodes
            total = sum(nodes)
            draft = torch.randint(0, 32000, (total,), generator=host)
            target = torch.randint(0, 32000, (total,), generator=host)
            first = torch.repeat_interleave(start[:-1], torch.tensor(nodes))
            agrees = (torch.rand(total, generator=host) < 0.7) & (parents >= 0)
            target[(first + parents.long())[agrees]] = draft[agrees]
            s["draft_tokens"], s["target_tokens"] = draft.cuda(), target.cuda()
    else:
        spans, kept = _spans(case)
        lens = _lens(case)
        dt = _DT[case["dtype"]]
        table, pool = _tables([a + b for a, b in zip(lens, spans)], case["block"], host)
        shape = (pool, case["block"], case["kv_heads"], case["dim"])
        make = lambda: torch.randn(shape, generator=dev, device="cuda", dtype=dt)  # noqa: E731
        s["key_caches"] = [make() for _ in range(case["layers"])]
        s["value_caches"] = [make() for _ in range(case["layers"])]
        s["block_tables"] = table.cuda()
        s["start_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        keep = torch.full((case["batch"], max(kept)), -1, dtype=torch.int32)
        for b, (n, k) in enumerate(zip(spans, kept)):
            head = min(case["head"], k)                       # the first tokens are always kept
            rest = torch.randperm(n - head, generator=host)[:k - head].sort().values + head
            keep[b, :k] = torch.cat([torch.arange(head), rest]).to(torch.int32)
        s["keep"] = keep.cuda()
        s["keep_lens"] = torch.tensor(kept, dtype=torch.int32).cuda()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rows(query_start, width):
    """Row of node i of sequence b as an array [batch, width], and which of them exist."""
    start = query_start.long()
    i = torch.arange(width, device=start.device)
    there = i[None, :] < (start[1:] - start[:-1])[:, None]
    return start[:-1, None] + i[None, :], there


def _pad(x, query_start, width, fill):
    """[T, ...] -> [batch, width, ...]."""
    rows, there = _rows(query_start, width)
    out = torch.full((rows.shape[0], width) + x.shape[1:], fill, dtype=x.dtype, device=x.device)
    out[there] = x[rows[there]]
    return out


def _unpad(x, query_start):
    """[batch, width, ...] -> [T, ...]."""
    _, there = _rows(query_start, x.shape[1])
    return x[there]


def _pad_parents(parents, query_start, width):
    return _pad(parents.long(), query_start, width, -2)     # -2: no such node


def _closure(parents):
    """bits[b, i, j]: j is i or an ancestor of i (products of the step matrix with itself)."""
    n = parents.shape[1]
    j = torch.arange(n, device=parents.device)
    step = ((parents[:, :, None] == j) | ((j[:, None] == j) & (parents > -2)[:, :, None])).float()
    reach = 1
    while reach < n:
        step = (torch.bmm(step, step) > 0).float()
        reach *= 2
    return step > 0


def _pack(bits):
    """Truth values [..., n] -> int32 words of 32, bit k of word w for value 32 w + k."""
    n = bits.shape[-1]
    words = -(-n // 32)
    bits = torch.nn.functional.pad(bits, (0, words * 32 - n)).unflatten(-1, (words, 32))
    value = (bits.long() << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(value >= 1 << 31, value - (1 << 32), value).to(torch.int32)


def _attend(s):
    q = _pad(s["query"].float(), s["query_start"], s["max_query_len"], 0.0)          # [B, n, Hq, D]
    words = _pad(s["tree_mask"].long(), s["query_start"], s["max_query_len"], 0)     # [B, n, W]
    lens = s["context_lens"].long()
    counts = (s["query_start"][1:] - s["query_start"][:-1]).long()
    pages = s["block_tables"].long().clamp(min=0)
    block, kv_heads = s["key_cache"].shape[1:3]
    batch, nodes, heads, dim = q.shape
    k = s["key_cache"][pages].float().flatten(1, 2)                                  # [B, L, Hkv, D]
    v = s["value_cache"][pages].float().flatten(1, 2)
    pos = torch.arange(k.shape[1], device=k.device)
    base = (lens - counts)[:, None, None]
    node = pos - base                                                                # [B, 1, L]
    inside = (node >= 0) & (node < counts[:, None, None])
    at = node.clamp(min=0, max=max(0, words.shape[2] * 32 - 1)).expand(batch, nodes, -1)
    seen = (words.gather(2, at // 32) >> (at % 32)) & 1
    mask = (pos < base) | (inside & (seen == 1))                                     # [B, n, L]
    group = heads // kv_heads
    q = q.view(batch, nodes, kv_heads, group, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [B, Hkv, G n, D]
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                          # [B, Hkv, G n, L]
    x = x.view(batch, kv_heads, group, nodes, -1)
    x = x.masked_fill(~mask[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = (x - top.clamp(min=-1e30)).exp()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).view(batch, kv_heads, group, nodes, dim)
    out = (out / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(batch, nodes, heads, dim)
    return _unpad(out, s["query_start"]).to(s["query"].dtype)


def _mask(s):
    parents = _pad_parents(s["parents"], s["query_start"], s["max_query_len"])
    bits = _closure(parents)
    counts = s["query_start"][1:] - s["query_start"][:-1]
    depth = bits.sum(-1) - 1
    position = (s["context_lens"] - counts).long()[:, None] + depth
    return _unpad(_pack(bits), s["query_start"]), _unpad(position, s["query_start"]).to(torch.int32)


def _accept(s):
    width = s["max_query_len"]
    parents = _pad_parents(s["parents"], s["query_start"], width)
    draft = _pad(s["draft_tokens"], s["query_start"], width, -1)
    target = _pad(s["target_tokens"], s["query_start"], width, -1)
    i = torch.arange(width, device=parents.device)
    # a node is confirmed if its parent's answer is its token and no earlier sibling was confirmed by it
    asked = (target.gather(1, parents.clamp(min=0)) == draft) & (parents >= 0)
    lowest = torch.full_like(parents, width).scatter_reduce(
        1, parents.clamp(min=0), torch.where(asked, i, torch.tensor(width, device=i.device)).expand_as(parents), "amin")
    confirmed = (asked & (lowest.gather(1, parents.clamp(min=0)) == i)) | ((i == 0) & (parents > -2))
    # it is accepted if every node above it is confirmed too
    accepted = ~(_closure(parents) & ~confirmed[:, None, :]).any(-1) & (parents > -2)
    lens = accepted.sum(-1)
    order = torch.where(accepted, i, torch.tensor(width, device=i.device)).sort(-1).values
    path = torch.where(i < lens[:, None], order, torch.tensor(-1, device=i.device))
    last = path.gather(1, (lens - 1).clamp(min=0)[:, None])
    following = torch.where(lens > 0, target.gather(1, last.clamp(min=0))[:, 0], torch.tensor(-1, device=i.device))
    return path.to(torch.int32), lens.to(torch.int32), following


def _compact(s):
    block = s["key_caches"][0].shape[1]
    keep = s["keep"].long()
    i = torch.arange(keep.shape[1], device=keep.device)
    there = i < s["keep_lens"][:, None]
    start = s["start_lens"].long()[:, None]

    def cell(position):
        position = torch.where(there, position, torch.zeros_like(position))
        return (s["block_tables"].long().gather(1, position // block) * block + position % block)[there]

    source, target = cell(start + keep), cell(start + i.expand_as(keep))
    for cache in s["key_caches"] + s["value_caches"]:
        flat = cache.view(-1, cache.shape[2] * cache.shape[3])
        flat[target] = flat[source]
    return s["key_caches"] + s["value_caches"]


def run(state):
    s = state
    if own:
        import paged_kv_cache_468_b200 as pkv
        if s["op"] == "attend":
            return pkv.paged_attention_tree(s["query"], s["query_start"], s["max_query_len"], s["tree_mask"], s["key_cache"],
                                            s["value_cache"], s["block_tables"], s["context_lens"], s["scale"])
        if s["op"] == "mask":
            return pkv.draft_tree_mask(s["parents"], s["query_start"], s["max_query_len"], s["context_lens"])
        if s["op"] == "accept":
            return pkv.draft_tree_accept(s["draft_tokens"], s["target_tokens"], s["parents"], s["query_start"], s["max_query_len"])
        pkv.kv_cache_compact(s["key_caches"], s["value_caches"], s["block_tables"], s["start_lens"], s["keep"], s["keep_lens"])
        return s["key_caches"] + s["value_caches"]
    return {"attend": _attend, "mask": _mask, "accept": _accept, "compact": _compact}[s["op"]](s)


# ---------------------------------------------------------------------------
# exact values
# ---------------------------------------------------------------------------
def exact(case, seed):
    """The definition, sequence by sequence, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] in ("mask", "accept"):
        return None                                # whole numbers: compared with the plain form itself
    table = s["block_tables"].cpu()
    if case["op"] == "compact":
        if case["layers"] * case["batch"] > 1024:
            return None
        out = []
        keep, count, start = s["keep"].cpu(), s["keep_lens"].tolist(), s["start_lens"].tolist()
        block = case["block"]
        for cache in s["key_caches"] + s["value_caches"]:
            before = cache.double()
            after = before.clone()
            for b in range(case["batch"]):
                old = start[b] + keep[b, :count[b]].long()
                new = start[b] + torch.arange(count[b])
                after[table[b, new // block].long().cuda(), (new % block).cuda()] = \
                    before[table[b, old // block].long().cuda(), (old % block).cuda()]
            out.append(after)
        return out
    starts, lens = s["query_start"].tolist(), s["context_lens"].tolist()
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    bits = ((s["tree_mask"].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1).flatten(1) == 1
    for b, total in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if hi == lo:
            continue
        n = hi - lo
        pages = table[b, :-(-total // case["block"])].long().cuda()
        k = s["key_cache"][pages].reshape(-1, case["kv_heads"], case["dim"])[:total].double()
        v = s["value_cache"][pages].reshape(-1, case["kv_heads"], case["dim"])[:total].double()
        visible = torch.cat([torch.ones(n, total - n, dtype=torch.bool, device="cuda"), bits[lo:hi, :n]], 1)
        for h in range(case["kv_heads"]):
            q = s["query"][lo:hi, h * group:(h + 1) * group].double()
            x = torch.einsum("ngd,ld->ngl", q, k[:, h]) * s["scale"]
            x = torch.where(visible[:, None], x, torch.full_like(x, float("-inf")))
            some = visible.any(1)[:, None, None]
            p = torch.where(some, torch.softmax(x, -1), torch.zeros_like(x))
            out[lo:hi, h * group:(h + 1) * group] = torch.einsum("ngl,ld->ngd", p, v[:, h])
    return out
