"""Random calls for drafted trees and eviction against the definitions: shapes, strides, masks and lengths as they come, each
call made twice with the same bits."""
import math
import random

import pytest
import torch

from attention_forward_prefill_gb300 import binding
from tests import evict_util
from tests.paged_util import Cache, assert_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(counts, start=0):
    cu = [start]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 0.7)), math.log(hi)))))))


def some_cache(rng, seed, longest):
    B, Hkv, G, d = spread(rng, 1, 12), rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16, 33]), rng.choice([64, 128])
    dtype = rng.choice([torch.float16, torch.bfloat16])
    top = spread(rng, 1, longest)
    lens = [rng.choice([top, rng.randint(0, top), spread(rng, 1, top)]) for _ in range(B)]
    cache = Cache(lens, Hkv, d, rng.choice([16, 32, 64, 128, 512]), dtype, slots_first=rng.random() < 0.5, seed=seed,
                  extra_cols=rng.choice([1, 2, 40]))
    return cache, lens, G * Hkv, G


@pytest.mark.parametrize("seed", range(16))
def test_trees(seed):
    rng = random.Random(seed)
    cache, lens, Hq, G = some_cache(rng, seed, 3000)
    most = spread(rng, 1, 120)
    counts = [rng.choice([0, 1, most, rng.randint(0, most)]) for _ in lens]
    total, ahead = sum(counts), rng.randint(0, 3)
    if total == 0:
        counts[0] = total = 1
    q = torch.randn(total + ahead, Hq, cache.d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(cache.dtype)
    words = -(-max(counts) // 32) + rng.randint(0, 2)
    mask = torch.randint(-1 << 31, 1 << 31, (total + ahead, words), device="cuda").to(torch.int32)
    args = (q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts, ahead)), max(counts) + rng.randint(0, 32 * words - max(counts)), mask)
    scale = rng.choice([None, 0.3, -0.1])
    lse = torch.full((total + ahead, Hq), 5.0, device="cuda")
    out = binding.prefill_tree(*args, scale=scale, lse=lse, out=torch.full_like(q, 3.0))
    again = binding.prefill_tree(*args, scale=scale, out=torch.full_like(q, 3.0))
    assert torch.equal(out, again) and (out[:ahead] == 3).all() and (lse[:ahead] == 5).all()
    t = ahead
    for b, n in enumerate(counts):
        if n:
            k, v = cache.keys(b)
            seen = evict_util.seen_of(mask[t:t + n], n, lens[b])
            want, want_lse, bound, off = evict_util.attend_seen(q[t:t + n].double(), k, v, scale or 1 / math.sqrt(cache.d), seen, cache.dtype)
            assert_rows(out[t:t + n], want, bound, f"sequence {b}")
            some = want_lse > -math.inf
            assert torch.equal(lse[t:t + n] > -math.inf, some)
            assert ((lse[t:t + n].double() - want_lse)[some].abs() <= off[some]).all()
        t += n


@pytest.mark.parametrize("seed", range(24))
def test_weights(seed):
    rng = random.Random(seed + 100)
    cache, lens, Hq, G = some_cache(rng, seed, 4000)
    B, Hkv, d = len(lens), cache.Hkv, cache.d
    one = rng.random() < 0.3
    most = 1 if one else spread(rng, 1, 700)
    counts = [1] * B if one else [rng.choice([0, 1, most, rng.randint(0, most)]) for _ in lens]
    if sum(counts) == 0:
        counts[0] = 1
    causal, scale, decay = rng.random() < 0.7, rng.choice([None, 0.2, -0.05]), rng.choice([1.0, 0.9])
    x = scale or 1 / math.sqrt(d)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(sum(counts), Hq, d, device="cuda", generator=g).to(cache.dtype)
    lse, seen, t = torch.empty(sum(counts), Hq, device="cuda"), [], 0
    for b, n in enumerate(counts):
        i = torch.arange(n, device="cuda")[:, None]
        see = torch.arange(lens[b], device="cuda") <= (lens[b] - n + i if causal else lens[b] + 0 * i)
        s = torch.einsum("nhgd,lhd->nhgl", q[t:t + n].double().view(n, Hkv, G, d), cache.keys(b)[0]) * x
        lse[t:t + n] = s.masked_fill(~see[:, None, None], -math.inf).logsumexp(-1).view(n, Hq).float()
        seen.append(see)
        t += n
    width = max(max(lens), 1) + rng.randint(0, 50)
    w = torch.rand(B, Hkv, width, device="cuda", generator=g) if rng.random() < 0.6 else None
    args = (q, lse, cache.k, cache.v, cache.table, cache.seq_lens, None if one and rng.random() < 0.5 else ints(offsets(counts)), max(counts))
    kw = dict(causal=causal, scale=scale, decay=decay)
    out = binding.cache_weigh(*args, weights=w, out=torch.full((B, Hkv, width), 7.0, device="cuda"), **kw)
    assert torch.equal(out, binding.cache_weigh(*args, weights=w, out=torch.full((B, Hkv, width), 7.0, device="cuda"), **kw))
    t = 0
    for b, n in enumerate(counts):
        want, bound = evict_util.weigh(q[t:t + n].double(), cache.keys(b)[0], lse[t:t + n].double(), x, seen[b])
        if w is not None:
            old = (decay if n else 1.0) * w[b, :, :lens[b]].double()
            want = want + old
            # the call takes decay as an fp32 number, off by at most 2^-24 of it (0.9 by 2^-25.2), and its product with
            # the old weight may round, by as much again; the sum's rounding is counted below
            bound = bound + (2 * 2.0 ** -24 * old if decay != 1.0 else 0.0)
        assert ((out[b, :, :lens[b]].double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all()
        assert (out[b, :, lens[b]:] == 7).all()
        t += n


@pytest.mark.parametrize("seed", range(10))
def test_selecting_and_moving(seed):
    rng = random.Random(seed + 200)
    cache, lens, _, _ = some_cache(rng, seed, 6000)
    B, Hkv = len(lens), cache.Hkv
    budget = spread(rng, 1, 2000)
    sink = rng.randint(0, budget)
    recent = rng.randint(0, budget - sink)
    heads, width = rng.choice([1, Hkv]), max(max(lens), 1) + rng.randint(0, 9)
    w = torch.rand(B, heads, width, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).pow(rng.choice([1, 8]))
    if rng.random() < 0.5:
        w = (w * 5).floor()
    keep, counts, kept = binding.cache_select(w, cache.seq_lens, budget, sink=sink, recent=recent)
    rows = w.cpu()
    lists = [[evict_util.select(rows[b, h].tolist(), lens[b], budget, sink, recent) for h in range(heads)] for b in range(B)]
    for b in range(B):
        for h in range(heads):
            mine = lists[b][h]
            assert keep[b, h].tolist() == mine + [-1] * (budget - len(mine))
            assert torch.equal(kept[b, h, :len(mine)].cpu(), rows[b, h, mine]) and not kept[b, h, len(mine):].any()
    want = [x.clone() for x in (cache.k, cache.v)]
    for x, old in zip(want, (cache.k, cache.v)):
        for b in range(B):
            for h in range(Hkv):
                src = torch.tensor(lists[b][h if heads > 1 else 0], dtype=torch.long, device="cuda")
                dst = torch.arange(len(src), device="cuda")
                table, S = cache.table[b].long(), cache.page
                x[table[dst // S], h, dst % S] = old[table[src // S], h, src % S]
    binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, keep, counts)
    for x, y in zip((cache.k, cache.v), want):
        assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


def test_two_captured_graphs_at_once():
    """Two graphs of weighed chunks and drafted trees, each with scratch of its own, replayed on two streams at a time."""
    made = []
    for i in range(2):
        cache = Cache([900, 333, 1500], 4, 64 if i else 128, 64, torch.float16, seed=i)
        counts = [200, 100, 64]
        cu = ints(offsets(counts))
        q = torch.randn(sum(counts), 16, cache.d, device="cuda").half()
        lse = torch.full((sum(counts), 16), 6.0, device="cuda")
        mask = torch.randint(-1 << 31, 1 << 31, (sum(counts), 7), device="cuda").to(torch.int32)
        bufs = [torch.zeros(3, 4, 1500, device="cuda"), torch.empty_like(q), torch.zeros_like(lse)]

        def step(bufs=bufs, cache=cache, cu=cu, q=q, lse=lse, mask=mask):
            binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, 200, out=bufs[0])
            binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, cu, 200, mask, out=bufs[1], lse=bufs[2])

        step()
        torch.cuda.synchronize()
        want = [x.clone() for x in bufs]
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for x in bufs:
            x.zero_()
        made.append((stream, graph, bufs, want))
    torch.cuda.synchronize()
    for _ in range(8):
        for stream, graph, _, _ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, bufs, want in made:
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))
