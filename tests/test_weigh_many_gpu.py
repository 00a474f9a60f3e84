"""Weighing for batches of more sequences than a CTA has threads, empty and idle ones among them."""
import math
import random

import pytest
import torch

from attention_forward_prefill_gb300 import binding
from tests import evict_util
from tests.paged_util import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


# up to 8 rows a kv head, more of them, and tensor-memory tiles (over 8 rows where there are many keys)
@pytest.mark.parametrize("B,most,Hq,Hkv,d", [(300, 1, 8, 2, 64), (1100, 2, 4, 1, 128), (257, 3, 40, 1, 64), (700, 5, 16, 4, 128), (1500, 9, 14, 2, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_sequences(B, most, Hq, Hkv, d, in_place):
    rng = random.Random(B)
    lens = [rng.choice([0, 1, 40, rng.randint(0, 400)]) if rng.random() < 0.7 else 0 for _ in range(B)]
    counts = [rng.randint(0, most) for _ in range(B)]
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    cache = Cache(lens, Hkv, d, 16, torch.float16, seed=B)
    g = torch.Generator(device="cuda").manual_seed(B)
    q = torch.randn(cu[-1], Hq, d, generator=g, device="cuda").half()
    lse = torch.full((cu[-1], Hq), 5.0, device="cuda")
    w = torch.rand(B, Hkv, 410, generator=g, device="cuda")
    old, out = w.clone(), w if in_place else torch.full_like(w, 7.0)
    binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, torch.tensor(cu, dtype=torch.int32, device="cuda"), most,
                        weights=w, out=out)
    worst = torch.zeros((), dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(zip(counts, lens)):
        behind = old[b, :, length:] if in_place else torch.full_like(old[b, :, length:], 7.0)
        assert torch.equal(out[b, :, length:], behind), b
        if length == 0:
            continue
        if n == 0:
            assert torch.equal(out[b, :, :length], old[b, :, :length]), b
            continue
        i = torch.arange(n, device="cuda")[:, None]
        seen = torch.arange(length, device="cuda") <= length - n + i
        want, bound = evict_util.weigh(q[cu[b]:cu[b + 1]].double(), cache.keys(b)[0], lse[cu[b]:cu[b + 1]].double(), 1 / math.sqrt(d), seen)
        want = want + old[b, :, :length].double()
        worst = torch.maximum(worst, ((out[b, :, :length].double() - want).abs() - bound - 2.0 ** -24 * want.abs()).max())
    assert worst <= 0
