"""Tree attention with values at both ends of bf16's range, in every kernel: an
output is an average of values, so it is finite however many keys there are and
however the weights are scaled while they are summed."""
import pytest
import torch

import paged_kv_cache_468_b200 as pkv
from tests import tree_util as tu

pytestmark = pytest.mark.gpu

# (heads, nodes, table columns): clusters of few and of more rows, few rows in
# parts, shares of one row tile, pairs of row tiles, transposed (head_dim 128)
FORMS = {"small clusters": ((2, 2), [2, 1], 0), "few parts": ((2, 2), [2, 1], 4096), "clusters": ((4, 1), [12, 30], 0),
         "shares": ((4, 1), [12, 30], 4096), "pairs": ((4, 1), [70, 30], 4096), "up to 64 rows": ((4, 1), [12, 16], 4096)}


def _case(form, D, gap, exponent, sign):
    """Keys whose scores step up by `gap` behind the first 128; positive values around 2^exponent."""
    (Hq, Hkv), nodes, columns = FORMS[form]
    bases = [700, 1300]
    c = tu.tree_case(nodes, bases, Hq, Hkv, D, 16, "bf16", seed=len(form) + D, columns=columns)
    g = torch.Generator().manual_seed(91)
    T = sum(nodes)
    c["query"] = (1 + 0.05 * torch.randn(T, Hq, D, generator=g)).to(torch.bfloat16)
    c["scale"] = sign * float(D) ** -0.5
    for b in range(2):
        L = nodes[b] + bases[b]
        k = 0.02 * torch.randn(L, Hkv, D, generator=g)
        k[128:] += sign * gap / D ** 0.5                   # scale x D x this = gap
        v = (1 + 0.9 * torch.rand(L, Hkv, D, generator=g)).to(torch.bfloat16).double() * 2.0 ** exponent
        c["keys"][b] = k.to(torch.bfloat16)
        c["values"][b] = v.to(torch.bfloat16)
        for j in range(L):
            page = int(c["block_tables"][b, j // 16])
            c["key_cache"][page, j % 16] = c["keys"][b][j]
            c["value_cache"][page, j % 16] = c["values"][b][j]
    return c


# 13 bits (9.2) and 7.6 bits (5.3): just below where the running maximum of the transposed and of the other
# kernels moves; 2^127: the largest binade; 2^-90: sums stay normal 32-bit numbers
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("gap", [0.0, 5.3, 9.2])
def test_values_of_any_size(form, D, gap):
    for exponent, sign in ((127, 1), (127, -1), (115, 1), (-90, 1)):
        c = _case(form, D, gap, exponent, sign)
        d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
        pkv.device_flags(clear=True)
        out = pkv.paged_attention_tree(d["query"], d["query_start"], d["max_query_len"], d["tree_mask"], d["key_cache"],
                                       d["value_cache"], d["block_tables"], d["context_lens"], d["scale"])
        assert pkv.device_flags() == 0
        assert torch.isfinite(out).all(), (exponent, sign)
        ref, tol = tu.attend_reference(c)
        over = (out.double().cpu() - ref).abs() - tol
        assert (over <= 0).all(), (exponent, sign, float((over / tol).max()) + 1)
