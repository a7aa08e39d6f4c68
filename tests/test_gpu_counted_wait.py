"""The tree attention kernels' wait, which counts its tries, gives up in time on
a barrier phase that nothing completes: the flag is set, the call returns and
the context stays usable."""
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from paged_kv_cache_468_b200 import pagedkv
from tests import tree_util as tu

pytestmark = pytest.mark.gpu


def test_counted_wait_runs_out_and_context_survives():
    pkv.device_flags(clear=True)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    pkv.selftest_counted_wait()
    end.record()
    assert pkv.device_flags(clear=True) == pagedkv.DEVFLAG_WAIT_TIMEOUT
    # 2^19 tries: long enough for any copy or product, short enough to end by itself
    ms = begin.elapsed_time(end)
    print(f"counted wait: {ms:.0f} ms")
    assert 200 < ms < 6000
    c = tu.tree_case([5, 9], [100, 30], 4, 2, 64, 16, "bf16", seed=1)
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    out = pkv.paged_attention_tree(d["query"], d["query_start"], d["max_query_len"], d["tree_mask"], d["key_cache"],
                                   d["value_cache"], d["block_tables"], d["context_lens"], d["scale"])
    ref, tol = tu.attend_reference(c)
    assert ((out.double().cpu() - ref).abs() <= tol).all()
    assert pkv.device_flags() == 0
