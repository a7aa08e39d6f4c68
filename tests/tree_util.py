"""Inputs and 64-bit references of the drafted-tree operators (shared by their
CPU and GPU tests).  The references are written from the definitions, sequence
by sequence, and share nothing with the library."""
from __future__ import annotations

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def random_parents(n, g, chain=False):
    """A tree whose node 0 is the root (a plain chain of nodes on request)."""
    if chain:
        return torch.arange(n, dtype=torch.int32) - 1
    p = [-1] + [int(torch.randint(max(0, i - 5), i, (1,), generator=g)) for i in range(1, n)]
    return torch.tensor(p[:n], dtype=torch.int32)


def ancestors(parents):
    """bits[i, j]: node j is i or an ancestor of i; depth[i]."""
    n = len(parents)
    bits, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for i in range(n):
        p = int(parents[i])
        if p >= 0:
            bits[i] = bits[p]
            depth[i] = depth[p] + 1
        bits[i, i] = True
    return bits, depth


def pack(bits, words):
    """[n, m] truth values -> int32 [n, words]."""
    out = np.zeros((bits.shape[0], words), dtype=np.uint32)
    for j in range(bits.shape[1]):
        out[:, j // 32] |= bits[:, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(out.view(np.int32).copy())


def accept(parents, draft, target):
    """(path, next token) of greedy verification."""
    if len(parents) == 0:
        return [], -1
    path = [0]
    while True:
        here = path[-1]
        following = [c for c in range(len(parents)) if int(parents[c]) == here and int(draft[c]) == int(target[here])]
        if not following:
            return path, int(target[here])
        path.append(following[0])


def tree_case(nodes, bases, Hq, Hkv, D, bs, dtype, seed, bits=None, q_scale=1.0, max_query_len=None, columns=0):
    """Drafted trees of `nodes[b]` nodes behind `bases[b]` committed tokens.  bits[b]: [n, n] truth
    values (default: a random tree's ancestors).  Cells that belong to no token hold NaN.  columns: the
    table's width at least (a wide table makes the library plan for long contexts)."""
    g = torch.Generator().manual_seed(seed)
    B = len(nodes)
    lens = [n + c for n, c in zip(nodes, bases)]
    pages = [-(-t // bs) for t in lens]
    NB = sum(pages) + 5
    order = torch.randperm(NB, generator=g).tolist()
    table = torch.full((B, max(1, columns, max(pages))), -1, dtype=torch.int32)
    kc = torch.full((NB, bs, Hkv, D), float("nan"))
    vc = torch.full((NB, bs, Hkv, D), float("nan"))
    ks, vs = [], []
    at = 0
    for b in range(B):
        ids = order[at:at + pages[b]]
        at += pages[b]
        table[b, :pages[b]] = torch.tensor(ids, dtype=torch.int32)
        k = torch.randn(lens[b], Hkv, D, generator=g).to(DT[dtype])
        v = torch.randn(lens[b], Hkv, D, generator=g).to(DT[dtype])
        ks.append(k)
        vs.append(v)
        for i, page in enumerate(ids):
            m = min(bs, lens[b] - i * bs)
            kc[page, :m] = k[i * bs:i * bs + m].float()
            vc[page, :m] = v[i * bs:i * bs + m].float()
    if bits is None:
        bits = [ancestors(random_parents(n, g))[0] for n in nodes]
    width = max_query_len or max(1, max(nodes))
    words = -(-width // 32)
    mask = torch.cat([pack(x, words) for x in bits])
    q = (torch.randn(sum(nodes), Hq, D, generator=g) * q_scale).to(DT[dtype])
    return dict(query=q, query_start=starts(nodes), max_query_len=width, tree_mask=mask,
                key_cache=kc.to(DT[dtype]), value_cache=vc.to(DT[dtype]), block_tables=table,
                context_lens=torch.tensor(lens, dtype=torch.int32), scale=float(D) ** -0.5,
                bits=bits, nodes=list(nodes), bases=list(bases), dtype=dtype, keys=ks, values=vs)


def attend_reference(c):
    """(out, tolerance), both float64 [T, Hq, D].

    The kernel rounds each weight p_j to the cache type (relative error at most
    half a step h = eps/2, normalised by the sum of the rounded weights), its
    output once more (h |out|), and works in 32 bits elsewhere:
      weights    h * sum_j p_j |v_j - out|
      output     h * |out|
      scores     a sum of D products has an error of at most D 2^-24 sum_d |q_d k_d|,
                 times |scale| (an error has no sign: with a negative scale the signed
                 factor took 2 d off the bound instead of adding it);
                 an error d in a score changes its weight by d relative, its share
                 and the normaliser by as much again: 2 d sum_j p_j |v_j|; 2^-20
                 covers the exponent's argument and the exponential itself
      sums       16 products at a time join a 32-bit accumulator (2^-23 each,
                 whichever way it rounds): (L / 16 + 16) 2^-23 sum_j p_j |v_j|
      f16        weights under 2^-14 are off by up to 2^-25 each, beside a
                 normaliser l (relative to the largest weight): L 2^-25 max|v| / l
    Second-order terms are covered by a factor of 1 + 2^-6."""
    h = torch.finfo(DT[c["dtype"]]).eps / 2
    T, Hq, D = c["query"].shape
    Hkv = c["key_cache"].shape[2]
    G = Hq // Hkv
    out, tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    row = 0
    for b, n in enumerate(c["nodes"]):
        base, L = c["bases"][b], c["bases"][b] + n
        k, v = c["keys"][b].double(), c["values"][b].double()
        seen = np.concatenate([np.ones((n, base), dtype=bool), c["bits"][b][:, :n]], axis=1)
        for i in range(n):
            idx = torch.from_numpy(np.nonzero(seen[i])[0])
            if len(idx) == 0:
                continue
            for head in range(Hq):
                q, kk, vv = c["query"][row + i, head].double(), k[idx, head // G], v[idx, head // G]
                x = (kk @ q) * c["scale"]
                w = torch.exp(x - x.max())
                p = w / w.sum()
                o = p @ vv
                d = D * 2.0 ** -24 * abs(c["scale"]) * float((kk.abs() @ q.abs()).max())
                absv = p @ vv.abs()
                t = h * o.abs() + h * (p @ (vv - o).abs()) + (2 * d + 2.0 ** -20 + (L / 16 + 16) * 2.0 ** -23) * absv
                if c["dtype"] == "f16":
                    t = t + L * 2.0 ** -25 * vv.abs().max() / w.sum() + 2.0 ** -25
                out[row + i, head], tol[row + i, head] = o, t * (1 + 2.0 ** -6)
        row += n
    return out, tol
