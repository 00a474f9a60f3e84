"""NaN and infinities among the values of drafted nodes: they reach the nodes that see them, may reach others of their sequence
(0 times infinity), and stay out of the other sequences and of the log-sum-exps."""
import math

import pytest
import torch

from attention_forward_prefill_gb300 import binding
from tests.paged_util import Cache

pytestmark = pytest.mark.gpu

# lens, nodes, query heads, kv heads, d: clusters, ranges, tensor-memory tiles
FORMS = [
    ([700, 40, 2000], [8, 5, 3], 32, 8, 128),
    ([9000, 300, 5000], [8, 5, 8], 16, 2, 128),
    ([1500, 90, 128], [33, 64, 17], 32, 8, 64),
]


@pytest.fixture(autouse=True)
def clean_status():
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


@pytest.mark.parametrize("form", FORMS, ids=["cluster", "ranges", "tiles"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf], ids=str)
def test_values_of_hidden_nodes(form, value):
    lens, counts, Hq, Hkv, d = form
    cache = Cache(lens, Hkv, d, 64, torch.bfloat16, seed=1)
    cu = torch.tensor([0, counts[0], counts[0] + counts[1], sum(counts)], dtype=torch.int32, device="cuda")
    q = torch.randn(sum(counts), Hq, d, device="cuda").bfloat16()
    # two branches from the context: even nodes and odd ones
    parents = torch.tensor(sum(([i - 2 if i > 1 else -1 for i in range(n)] for n in counts), []), dtype=torch.int32, device="cuda")
    mask, _ = binding.tree_mask(parents, cu, max(counts))

    def run():
        lse = torch.empty(sum(counts), Hq, device="cuda")
        return binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(counts), mask, lse=lse), lse

    out, lse = run()
    at = lens[1] - counts[1] + 1  # node 1 of the middle sequence
    cache.v[int(cache.table[1, at // 64]), :, at % 64] = value
    got, got_lse = run()
    assert torch.equal(got_lse, lse)
    a, z = counts[0], counts[0] + counts[1]
    assert torch.equal(got[:a], out[:a]) and torch.equal(got[z:], out[z:])
    assert not torch.isfinite(got[a + 1:z:2]).any()  # the nodes behind it, and itself
