"""Weighing where some sequences have no query tokens: their pages and keys are not asked for, and their weights stay as they
are, whichever kernel runs."""
import math

import pytest
import torch

from attention_forward_prefill_gb300 import binding
from tests import evict_util
from tests.paged_util import Cache

pytestmark = pytest.mark.gpu

# (query tokens, query heads, kv heads, d): up to 8 rows a kv head, some more of them, and tensor-memory tiles
KERNELS = [([0, 1, 0], 8, 2, 64), ([0, 5, 0], 32, 8, 128), ([0, 60, 0], 32, 8, 128), ([0, 70, 0], 14, 2, 64)]
LENS = [700, 300, 131]


@pytest.fixture(autouse=True)
def clean_status():
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def step(counts, Hq, Hkv, d):
    cache = Cache(LENS, Hkv, d, 64, torch.float16, seed=d)
    g = torch.Generator(device="cuda").manual_seed(Hq)
    q = torch.randn(sum(counts), Hq, d, generator=g, device="cuda").half()
    lse = torch.full((sum(counts), Hq), 6.0, device="cuda")
    w = torch.rand(3, Hkv, 750, generator=g, device="cuda")
    cu = ints([0, counts[0], counts[0] + counts[1], sum(counts)])
    return cache, q, lse, w, cu


def check_active(cache, q, lse, w, out, counts, decay):
    k, n, length = cache.keys(1)[0], counts[1], LENS[1]
    i = torch.arange(n, device="cuda")[:, None]
    seen = torch.arange(length, device="cuda") <= length - n + i
    want, bound = evict_util.weigh(q.double(), k, lse.double(), 1 / math.sqrt(cache.d), seen)
    want = want + decay * w[1, :, :length].double()
    assert ((out[1, :, :length].double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("counts,Hq,Hkv,d", KERNELS)
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_of_idle_sequences_are_not_asked_for(counts, Hq, Hkv, d, in_place):
    """Rows of the table that are no pages: nothing is recorded, and the weights are there."""
    cache, q, lse, w, cu = step(counts, Hq, Hkv, d)
    table = cache.table.clone()
    table[0], table[2] = -1, 1 << 30
    old = w.clone()
    out = w if in_place else torch.full_like(w, 7.0)
    binding.cache_weigh(q, lse, cache.k, cache.v, table, cache.seq_lens, cu, max(counts), weights=w, decay=0.5, out=out)
    assert binding.fa_device_status(True) == 0
    for b in (0, 2):
        assert torch.equal(out[b, :, :LENS[b]], old[b, :, :LENS[b]])
    for b, n in enumerate(LENS):
        assert torch.equal(out[b, :, n:], old[b, :, n:] if in_place else torch.full_like(old[b, :, n:], 7.0))
    check_active(cache, q, lse, old, out, counts, 0.5)


@pytest.mark.parametrize("counts,Hq,Hkv,d", KERNELS)
def test_idle_sequences_of_a_first_call_have_zeros(counts, Hq, Hkv, d):
    cache, q, lse, w, cu = step(counts, Hq, Hkv, d)
    table = cache.table.clone()
    table[0], table[2] = -1, -1
    out = torch.full_like(w, 7.0)
    binding.cache_weigh(q, lse, cache.k, cache.v, table, cache.seq_lens, cu, max(counts), out=out)
    for b in (0, 2):
        assert not out[b, :, :LENS[b]].any()
    check_active(cache, q, lse, torch.zeros_like(w), out, counts, 1.0)


@pytest.mark.parametrize("counts,Hq,Hkv,d", KERNELS)
def test_pages_of_sequences_with_tokens_are_checked(counts, Hq, Hkv, d):
    cache, q, lse, w, cu = step(counts, Hq, Hkv, d)
    table = cache.table.clone()
    table[1, 2] = -1
    binding.cache_weigh(q, lse, cache.k, cache.v, table, cache.seq_lens, cu, max(counts), weights=w, out=w)
    assert binding.fa_device_status(True) == binding.FA_ERR_PAGE


@pytest.mark.parametrize("counts,Hq,Hkv,d", KERNELS)
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_of_idle_sequences_keep_their_bits(counts, Hq, Hkv, d, in_place):
    """-0, NaN of any bits, infinities and subnormals too."""
    cache, q, lse, w, cu = step(counts, Hq, Hkv, d)
    some = ints([-(1 << 31), 0, 0x7fc12345, 0x7f800000, -0x800000, 1, -0x7fffffff, 0x3f800000])
    pick = torch.randint(0, 8, w.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    w.copy_(some[pick].view(torch.float32))
    old = w.clone().view(torch.int32)
    out = w if in_place else torch.full_like(w, 7.0)
    binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(counts), weights=w, decay=0.5, out=out)
    for b in (0, 2):
        assert torch.equal(out[b, :, :LENS[b]].contiguous().view(torch.int32), old[b, :, :LENS[b]])
