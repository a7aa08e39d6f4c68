"""Small tree-attention calls (a cluster per item, parts joined in shared
memory) launched many times: every launch gives the first one's bits, no wait
runs out, and the first agrees with the 64-bit reference."""
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from tests import tree_util as tu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("nodes,bases", [([9], [500]), ([5, 0, 17], [130, 20, 0]), ([20] * 40, list(range(0, 400, 10)))])
def test_cluster_launches_repeat(D, bs, nodes, bases):
    c = tu.tree_case(nodes, bases, 4, 1, D, bs, "bf16", seed=D + len(nodes))
    assert pkv.tree_workspace_bytes(len(nodes), c["max_query_len"], sum(nodes), 4, 1, D, c["block_tables"].shape[1], bs) == 0
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    pkv.device_flags(clear=True)
    outs = [torch.full_like(d["query"], 3.0) for _ in range(300)]
    for out in outs:
        pkv.paged_attention_tree(d["query"], d["query_start"], d["max_query_len"], d["tree_mask"], d["key_cache"],
                                 d["value_cache"], d["block_tables"], d["context_lens"], d["scale"], out=out)
    assert pkv.device_flags() == 0
    assert all(torch.equal(out, outs[0]) for out in outs)
    ref, tol = tu.attend_reference(c)
    assert ((outs[0].double().cpu() - ref).abs() <= tol).all()
