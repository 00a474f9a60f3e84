"""Query rows that weigh nothing, their log-sum-exp being infinite, whatever their queries hold: those of padding, say."""
import math

import pytest
import torch

from attention_forward_prefill_gb300 import binding
from tests import evict_util
from tests.paged_util import Cache

pytestmark = pytest.mark.gpu

# lens, query tokens, query heads, kv heads, d: up to 8 rows a kv head, more of them, and tensor-memory tiles
FORMS = [
    ([500, 77], [1, 1], 32, 8, 128),
    ([500, 77], [5, 3], 32, 8, 64),
    ([900, 300], [400, 300], 32, 8, 128),
    ([900, 300, 40], [500, 300, 90], 14, 2, 64),   # chunks of 126 rows
    ([700], [520], 50, 2, 128),                    # of 125
]


@pytest.fixture(autouse=True)
def clean_status():
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 1.0], ids=str)
@pytest.mark.parametrize("none", [-math.inf, math.inf], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_rows_left_out(form, value, none, causal):
    lens, counts, Hq, Hkv, d = form
    cache = Cache(lens, Hkv, d, 64, torch.bfloat16, seed=1)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(sum(counts), Hq, d, generator=g, device="cuda").bfloat16()
    lse = torch.rand(sum(counts), Hq, generator=g, device="cuda") + 6
    out_of_it = torch.rand(lse.shape, generator=g, device="cuda") < 0.3
    out_of_it[-1, 0], out_of_it[0, -1] = True, False
    scale, t, want = 1 / math.sqrt(d), 0, []
    for b, n in enumerate(counts):
        i = torch.arange(n, device="cuda")[:, None]
        seen = torch.arange(lens[b], device="cuda") <= (lens[b] - n + i if causal else lens[b] + 0 * i)
        rest = lse[t:t + n].double().masked_fill(out_of_it[t:t + n], -math.inf)  # (which adds nothing to the definition either)
        want.append(evict_util.weigh(q[t:t + n].double(), cache.keys(b)[0], rest, scale, seen))
        t += n
    q[out_of_it] = value
    lse[out_of_it] = none
    got = torch.full((len(lens), Hkv, max(lens)), 7.0, device="cuda")
    binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, offsets(counts), max(counts), causal=causal, out=got)
    for b, n in enumerate(lens):
        p, bound = want[b]
        assert ((got[b, :, :n].double() - p).abs() <= bound + 2.0 ** -24 * p).all(), b
        assert (got[b, :, n:] == 7).all()


@pytest.mark.parametrize("form", FORMS, ids=str)
def test_rows_with_a_finite_sum_still_pass_nan_on(form):
    lens, counts, Hq, Hkv, d = form
    cache = Cache(lens, Hkv, d, 64, torch.float16, seed=1)
    q = torch.randn(sum(counts), Hq, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    lse = torch.full((sum(counts), Hq), 6.0, device="cuda")
    lse[:, 0] = -math.inf
    q[0, 1] = math.nan   # a row of the first sequence and kv head that counts
    lse[0, Hq // Hkv] = math.nan   # and one of the second
    got = binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, offsets(counts), max(counts))
    sees = lens[0] - counts[0] + 1
    assert torch.isnan(got[0, :2, :sees]).all() and not torch.isnan(got[0, :2, sees:]).any()
    assert not torch.isnan(got[0, 2:]).any() and not torch.isnan(got[1:]).any()
