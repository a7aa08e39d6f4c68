"""Refusals of the drafted-tree calls on the host, the allocator's truncate, and
the references themselves (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from paged_kv_cache_468_b200 import pagedkv
from tests import tree_util as tu

A16 = 0x10000


def test_mask_host_validation():
    L = pkv.lib()

    def call(p=A16, T=8, qs=A16, mql=8, cl=A16, B=2, mask=A16, pos=A16):
        return L.pkv_draft_tree_mask(p, T, qs, mql, cl, B, mask, pos, None)
    assert call(T=-1) == pagedkv.ERR_INVALID_ARG
    assert call(mql=-1) == pagedkv.ERR_INVALID_ARG
    assert call(mql=1025) == pagedkv.ERR_UNSUPPORTED
    assert call(B=65536) == pagedkv.ERR_UNSUPPORTED
    assert call(p=None) == pagedkv.ERR_INVALID_ARG
    assert call(mask=A16 + 2) == pagedkv.ERR_MISALIGNED
    assert call(B=0, p=None, mask=None) == pagedkv.OK
    assert call(T=0, p=None, mask=None) == pagedkv.OK


def test_accept_host_validation():
    L = pkv.lib()

    def call(d=A16, t=A16, p=A16, T=8, qs=A16, mql=8, B=2, path=A16, lens=A16, nxt=A16):
        return L.pkv_draft_tree_accept(d, t, p, T, qs, mql, B, path, lens, nxt, None)
    assert call(T=-1) == pagedkv.ERR_INVALID_ARG
    assert call(mql=1025) == pagedkv.ERR_UNSUPPORTED
    assert call(d=None) == pagedkv.ERR_INVALID_ARG
    assert call(path=None) == pagedkv.ERR_INVALID_ARG
    assert call(d=A16 + 4) == pagedkv.ERR_MISALIGNED
    assert call(nxt=A16 + 4) == pagedkv.ERR_MISALIGNED
    assert call(lens=A16 + 2) == pagedkv.ERR_MISALIGNED
    assert call(B=0, d=None, lens=None) == pagedkv.OK


def test_tree_attention_host_validation():
    L = pkv.lib()

    def call(q=A16, T=64, qs=A16, mql=32, mask=A16, kc=A16, vc=A16, bt=A16, mb=8, cl=A16, B=2, Hq=8, Hkv=2, D=128,
             bs=16, nb=100, scale=0.125, ws=A16, wsb=1 << 40, out=A16, dt=1):
        return L.pkv_paged_attention_tree(q, T, qs, mql, mask, kc, vc, bt, mb, cl, B, Hq, Hkv, D, bs, nb, scale, ws, wsb,
                                          out, dt, None)
    assert call(Hq=32, Hkv=2) == pagedkv.ERR_UNSUPPORTED           # group 16 > 8
    assert call(D=96) == pagedkv.ERR_UNSUPPORTED
    assert call(bs=8) == pagedkv.ERR_UNSUPPORTED
    assert call(mql=1025) == pagedkv.ERR_UNSUPPORTED
    assert call(dt=7) == pagedkv.ERR_INVALID_ARG
    assert call(T=-1) == pagedkv.ERR_INVALID_ARG
    assert call(nb=0) == pagedkv.ERR_INVALID_ARG
    assert call(nb=1 << 27) == pagedkv.ERR_INVALID_ARG             # num_blocks * block_size = 2^31
    assert call(scale=float("nan")) == pagedkv.ERR_INVALID_ARG
    assert call(scale=3.4e38) == pagedkv.ERR_INVALID_ARG          # (times log2 e it is infinite)
    assert call(mask=None) == pagedkv.ERR_INVALID_ARG
    assert call(q=A16 + 8) == pagedkv.ERR_MISALIGNED
    assert call(mask=A16 + 2) == pagedkv.ERR_MISALIGNED
    assert call(B=0, q=None, out=None) == pagedkv.OK
    assert call(T=0, q=None, out=None) == pagedkv.OK
    assert pkv.tree_workspace_bytes(2, 32, 64, 8, 2, 128, 8, 16) == 0      # a small call: no workspace
    need = pkv.tree_workspace_bytes(2, 32, 64, 8, 2, 128, 4096, 16)
    assert need > 0
    assert call(mb=4096, ws=None) == pagedkv.ERR_WORKSPACE
    assert call(mb=4096, wsb=need - 1) == pagedkv.ERR_WORKSPACE
    assert call(mb=4096, ws=A16 + 8) == pagedkv.ERR_MISALIGNED
    assert pkv.tree_workspace_bytes(2, 32, 64, 8, 2, 96, 4096, 16) == 0    # a shape that the call refuses
    # more units than a call counts: 60000 sequences x 8 kv heads x 32 row tiles x 256 key tiles
    assert pkv.tree_workspace_bytes(60000, 512, 64, 64, 8, 128, 1024, 16) == 0
    assert call(B=60000, T=1 << 20, mql=512, Hq=64, Hkv=8, mb=1024) == pagedkv.ERR_UNSUPPORTED


def test_compact_host_validation():
    L = pkv.lib()

    def call(caches=(A16, 2 * A16), values=(3 * A16, 4 * A16), n=2, bt=A16, mb=8, st=A16, kp=A16, K=500, kl=A16, B=2, Hkv=2,
             D=64, nb=100, bs=16, ws=A16, wsb=1 << 40, dt=1):
        arr = ctypes.c_void_p * 2
        return L.pkv_kv_cache_compact(arr(*caches) if caches else None, arr(*values), n, bt, mb, st, kp, K, kl, B, Hkv, D,
                                      nb, bs, ws, wsb, dt, None)
    assert call(n=-1) == pagedkv.ERR_INVALID_ARG
    assert call(mb=0) == pagedkv.ERR_INVALID_ARG
    assert call(K=-1) == pagedkv.ERR_INVALID_ARG
    assert call(D=12) == pagedkv.ERR_UNSUPPORTED
    assert call(B=65536) == pagedkv.ERR_UNSUPPORTED
    assert call(dt=3) == pagedkv.ERR_INVALID_ARG
    assert call(nb=1 << 31) == pagedkv.ERR_INVALID_ARG
    assert call(mb=1 << 26) == pagedkv.ERR_INVALID_ARG
    assert call(caches=None) == pagedkv.ERR_INVALID_ARG
    assert call(caches=(A16, None)) == pagedkv.ERR_INVALID_ARG
    assert call(caches=(A16, A16 + 8)) == pagedkv.ERR_MISALIGNED
    assert call(kp=A16 + 2) == pagedkv.ERR_MISALIGNED
    assert call(n=0, caches=None) == pagedkv.OK
    assert call(B=0, bt=None) == pagedkv.OK
    assert call(K=0, kp=None) == pagedkv.OK
    need = pkv.compact_workspace_bytes(2, 2, 500, 2, 64)
    assert need > 0 and pkv.compact_workspace_bytes(2, 2, 100, 2, 64) == 0
    assert call(ws=None) == pagedkv.ERR_WORKSPACE
    assert call(wsb=need - 1) == pagedkv.ERR_WORKSPACE
    assert call(ws=A16 + 2) == pagedkv.ERR_MISALIGNED
    assert call(K=(1 << 30) - 1, mb=1 << 25, B=60000) == pagedkv.ERR_UNSUPPORTED   # chunks past 2^31


def test_binding_refuses_wrong_tensors():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        pkv.draft_tree_mask(i(4), i(3), 4, i(2))                       # CPU tensors
    with pytest.raises(ValueError):
        pkv.draft_tree_mask(i(4).long(), i(3), 4, i(2))
    with pytest.raises(ValueError):
        pkv.draft_tree_mask(i(4), i(3), 1025, i(2))
    with pytest.raises(ValueError):
        pkv.draft_tree_mask(i(4), i(3), 4, i(3))                       # lengths of another batch
    with pytest.raises(ValueError):
        pkv.draft_tree_accept(i(4), i(4), i(4), i(3), 4)               # tokens are int64
    q, c = torch.zeros(4, 8, 64, dtype=torch.float16), torch.zeros(4, 16, 8, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pkv.paged_attention_tree(q, i(3), 40, i(4, 1), c, c.clone(), i(2, 2), i(2), 0.1)   # the mask wants 2 words
    with pytest.raises(ValueError):
        pkv.paged_attention_tree(q, i(3), 4, i(4, 1), c, c.clone(), i(2, 2), i(2), 0.1)    # CPU tensors
    with pytest.raises(ValueError):
        pkv.kv_cache_compact([], [], i(2, 2), i(2), i(2, 3), i(2))
    with pytest.raises(ValueError):
        pkv.kv_cache_compact([c], [c, c], i(2, 2), i(2), i(2, 3), i(2))


def test_truncate_releases_the_tail():
    a = pkv.BlockAllocator(20, 16, shuffle_seed=1)
    t = a.new_seq(100)                                                 # 7 blocks
    first = list(t)
    a.truncate(t, 100)
    assert t == first and a.num_free == 13
    a.truncate(t, 33)
    assert t == first[:3] and a.num_free == 17
    other = a.fork(t)
    a.truncate(t, 32)                                                  # the shared block lives on
    assert t == first[:2] and a.num_free == 17 and a.refcount(first[2]) == 1
    a.truncate(other, 16)
    assert a.num_free == 18
    a.truncate(t, 0)
    assert t == [] and a.num_free == 19 and a.refcount(first[0]) == 1
    with pytest.raises(pkv.PagedKVError):
        a.truncate(other, -1)
    with pytest.raises(pkv.PagedKVError):
        a.truncate([first[0], first[5]], 16)                           # a block that is already free
    assert a.refcount(first[0]) == 1 and a.num_free == 19


def test_references_agree_with_a_hand_worked_tree():
    #      0
    #     / \
    #    1   2
    #    |   | \
    #    3   4  5
    parents = [-1, 0, 0, 1, 2, 2]
    bits, depth = tu.ancestors(parents)
    assert depth.tolist() == [0, 1, 1, 2, 2, 2]
    assert np.nonzero(bits[4])[0].tolist() == [0, 2, 4] and np.nonzero(bits[3])[0].tolist() == [0, 1, 3]
    assert tu.pack(bits, 1)[:, 0].tolist() == [1, 3, 5, 11, 21, 37]
    assert tu.accept(parents, [9, 4, 7, 1, 8, 8], [7, 0, 8, 0, 6, 5]) == ([0, 2, 4], 6)
    assert tu.accept(parents, [9, 4, 7, 1, 8, 8], [3, 0, 8, 0, 6, 5]) == ([0], 3)
