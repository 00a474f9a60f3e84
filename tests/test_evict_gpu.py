"""Eviction on the GPU: accumulated weights against the definition in 64 bits, selections and moved tokens against plain
Python, all of them in use together, in CUDA graphs and on other streams, faults on the device."""
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


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(counts, start=0):
    cu = [start]
    for n in counts:
        cu.append(cu[-1] + n)
    return cu


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---------------------------------------------------------------- weights
# (lens, query tokens or None for one each, query heads, kv heads, d, page, dtype, slots first)
FORMS = [
    ([1000], None, 12, 12, 64, 16, torch.float16, False),
    ([1, 17, 128, 129, 5000], None, 32, 8, 128, 64, torch.bfloat16, False),
    ([300, 0, 40], None, 14, 2, 64, 16, torch.float16, True),
    ([16, 1], [16, 1], 4, 4, 128, 16, torch.bfloat16, False),
    ([700, 64, 300, 0], [9, 64, 0, 3], 8, 2, 64, 32, torch.float16, False),
    ([3000, 250], [33, 200], 16, 16, 128, 128, torch.bfloat16, True),
    ([1500, 777, 2100], [400, 300, 129], 32, 8, 128, 64, torch.bfloat16, False),
    ([2600, 513], [1024, 513], 14, 2, 64, 16, torch.float16, True),
    ([100, 4], [300, 9], 6, 2, 128, 64, torch.float16, False),   # more query tokens than keys
    ([257], [255], 130, 1, 64, 256, torch.bfloat16, False),
    ([70, 33] * 40, [2, 1] * 40, 64, 8, 128, 32, torch.bfloat16, False),
    ([1000, 40, 513] * 10, [5, 8, 1] * 10, 32, 8, 128, 64, torch.bfloat16, False),   # few rows, many keys
    ([2000, 1, 600] * 12, [6, 1, 3] * 12, 14, 2, 64, 16, torch.float16, True),
    ([900, 640], [500, 640], 50, 2, 128, 64, torch.bfloat16, False),   # 125 rows of a chunk
    ([700, 129], [300, 20], 70, 2, 64, 32, torch.float16, False),      # 105
    ([400], [130], 66, 1, 128, 128, torch.bfloat16, False),            # 66
]


def prepared(form, causal, scale, seed=0, behind=float("nan")):
    lens, counts, Hq, Hkv, d, page, dtype, slots_first = form
    cache = Cache(lens, Hkv, d, page, dtype, slots_first=slots_first, seed=seed, behind=behind)
    news = counts or [1] * len(lens)
    q = (torch.randn(sum(news), Hq, d, generator=generator(seed + 1), device="cuda") * 1.5).to(dtype)
    lse, seen, t = torch.empty(sum(news), Hq, device="cuda"), [], 0
    for n, length, (k, _) in zip(news, lens, (cache.keys(b) for b in range(len(lens)))):
        i = torch.arange(n, device="cuda")[:, None]
        see = torch.arange(length, device="cuda") <= (length - n + i if causal else length + 0 * i)
        x = torch.einsum("nhgd,lhd->nhgl", q[t:t + n].double().view(n, Hkv, Hq // Hkv, d), k) * scale
        lse[t:t + n] = x.masked_fill(~see[:, None, None], -math.inf).logsumexp(-1).view(n, Hq).float()
        seen.append(see)
        t += n
    return cache, q, lse, seen, news


def check_weights(form, cache, q, lse, seen, news, scale, weights, decay, out, before):
    lens, t = form[0], 0
    for b, (n, length) in enumerate(zip(news, lens)):
        k, _ = cache.keys(b)
        got = out[b, :, :length].double()
        want, bound = evict_util.weigh(q[t:t + n].double(), k, lse[t:t + n].double(), scale, seen[b])
        if weights is not None:
            want = want + (decay if n else 1.0) * weights[b, :, :length].double()
        err = (got - want).abs()
        tol = bound + 2.0 ** -24 * want.abs()
        assert (err <= tol).all(), f"sequence {b}: {float((err - tol).max())} over at {int((err - tol).argmax())}, " \
                                   f"{int((err > tol).sum())} of {err.numel()}"
        assert torch.equal(out[b, :, length:], before[b, :, length:])
        t += n


def run_weigh(form, causal=True, scale=None, weights=True, decay=0.75, width=None, **more):
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    scale = 1 / math.sqrt(d) if scale is None else scale
    cache, q, lse, seen, news = prepared(form, causal, scale)
    width = width or max(lens) + 3
    w = torch.rand(len(lens), Hkv, width, generator=generator(5), device="cuda") * 3 if weights else None
    out = torch.full((len(lens), Hkv, width), 7.0, device="cuda")
    cu = None if counts is None else ints(offsets(counts))
    got = binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(news), causal=causal, scale=scale,
                              weights=w, decay=decay, out=out, **more)
    assert got is out
    check_weights(form, cache, q, lse, seen, news, scale, w, decay, out, torch.full_like(out, 7.0))
    return cache, q, lse, cu, news, w, out


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{str(f[0])[:24]}-{str(f[1])[:20]}-{f[2]}over{f[3]}x{f[4]}")
@pytest.mark.parametrize("causal", [True, False])
def test_weigh(form, causal):
    run_weigh(form, causal)


@pytest.mark.parametrize("form", [FORMS[1], FORMS[6], FORMS[7]], ids=["tokens", "chunks", "chunks64"])
@pytest.mark.parametrize("kw", [dict(scale=-0.15), dict(scale=0.0), dict(weights=False), dict(decay=0.0), dict(decay=-1.5),
                                dict(scale=1.0)], ids=str)
def test_weigh_scales_and_decays(form, kw):
    run_weigh(form, **kw)


@pytest.mark.parametrize("form", [FORMS[1], FORMS[6], FORMS[7], FORMS[10]], ids=["tokens", "chunks", "chunks64", "many"])
def test_weigh_in_place_new_and_again(form):
    cache, q, lse, cu, news, w, out = run_weigh(form)
    args = (q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(news))
    again = torch.full_like(out, 7.0)
    binding.cache_weigh(*args, weights=w, decay=0.75, out=again)
    assert torch.equal(again, out)
    fresh = binding.cache_weigh(*args, weights=w, decay=0.75)
    kept = w.clone()
    assert binding.cache_weigh(*args, weights=w, decay=0.75, out=w) is w
    for b, n in enumerate(form[0]):
        assert torch.equal(w[b, :, :n], out[b, :, :n]) and torch.equal(w[b, :, n:], kept[b, :, n:])
        assert torch.equal(fresh[b, :, :n], out[b, :, :n]) and not fresh[b, :, n:].any()
    assert binding.cache_weigh(*args).shape == (len(form[0]), form[3], cache.table.shape[1] * cache.page)


def test_weights_of_a_prefill_add_up_to_its_rows():
    """With the log-sum-exp that prefill_paged returns, a row's weights add up to 1."""
    lens, counts, Hq, Hkv, d, page, dtype, _ = form = FORMS[6]
    cache, q, _, _, news = prepared(form, True, 1 / math.sqrt(d))
    lse = torch.empty(sum(news), Hq, device="cuda")
    cu = ints(offsets(counts))
    binding.prefill_paged(q, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(news), causal=True, lse=lse)
    w = binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(news))
    for b, n in enumerate(counts):
        rows = n * Hq // Hkv
        # prefill's sum adds weights rounded to bf16
        assert ((w[b].double().sum(-1) - rows).abs() <= rows * (2.0 ** -8 + 2.0 ** -12)).all()


@pytest.mark.parametrize("form", [FORMS[1], FORMS[6], FORMS[7]], ids=["tokens", "chunks", "chunks64"])
def test_weigh_non_finite(form):
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    cache, q, lse, cu, news, w, out = run_weigh(form)
    args = (cache.k, cache.v, cache.table, cache.seq_lens, cu, max(news))
    # a key of NaN reaches its own weight alone
    b, at = 1, 9
    where = (int(cache.table[b, at // page]), 0, at % page)
    old = cache.k[where].clone()
    cache.k[where] = math.nan
    got = binding.cache_weigh(q, lse, *args, weights=w, decay=0.75, out=torch.full_like(out, 7.0))
    assert torch.isnan(got[b, 0, at])
    got[b, 0, at] = out[b, 0, at]
    assert torch.equal(got, out)
    cache.k[where] = old
    # a row that saw nothing adds nothing, whatever its query holds but NaN; one of NaN reaches what it sees
    q2, lse2 = q.clone(), lse.clone()
    lse2[0] = -math.inf
    got = binding.cache_weigh(q2, lse2, *args, weights=w, decay=0.75, out=torch.full_like(out, 7.0))
    check_weights(form, cache, q, lse2, [torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n) for n, m in zip(news, lens)],
                  news, 1 / math.sqrt(d), w, 0.75, got, torch.full_like(out, 7.0))
    lse2[0, 0] = math.nan
    got = binding.cache_weigh(q2, lse2, *args, weights=w, decay=0.75, out=torch.full_like(out, 7.0))
    sees = lens[0] - news[0] + 1
    assert torch.isnan(got[0, 0, :sees]).all() and not torch.isnan(got[0, 0, sees:]).any() and not torch.isnan(got[0, 1:]).any()


def test_weigh_far_pages_wide_rows_and_faults():
    """Pages and weights behind 2^32 elements; lengths and pages out of range."""
    form = ([300, 140], [2, 90], 4, 2, 128, 64, torch.float16, False)
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    cache = Cache(lens, Hkv, d, page, dtype, total_pages=(1 << 32) // (Hkv * d * page) + 9, behind=0.0)
    scale = 1 / math.sqrt(d)
    _, q, lse, seen, news = prepared(form, True, scale)  # (the same keys: the same seed)
    seen = [torch.ones(n, m, dtype=torch.bool, device="cuda").tril(m - n) for n, m in zip(counts, lens)]
    width = (1 << 30) - 64
    out = torch.zeros(2, Hkv, width, device="cuda")
    args = (q, lse, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts)), max(counts))
    binding.cache_weigh(*args, out=out)
    for b, n in enumerate(lens):
        k, _ = cache.keys(b)
        t = sum(counts[:b])
        want, bound = evict_util.weigh(q[t:t + counts[b]].double(), k, lse[t:t + counts[b]].double(), scale, seen[b])
        assert ((out[b, :, :n].double() - want).abs() <= bound + 2.0 ** -24 * want).all()
        assert not out[b, :, n:n + 1000].any()
    del out
    binding.cache_weigh(*args[:5], ints([301, 140 + 1000]), *args[6:])
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN
    short = torch.zeros(2, Hkv, 299, device="cuda")
    binding.cache_weigh(*args, out=short)
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN
    bad = cache.table.clone()
    bad[1, 1] = -1
    got = binding.cache_weigh(*args[:4], bad, *args[5:])
    assert binding.fa_device_status(True) == binding.FA_ERR_PAGE
    zero = torch.zeros_like(cache.keys(1)[0])
    want, bound = evict_util.weigh(q[2:].double(), zero, lse[2:].double(), scale, seen[1])
    assert ((got[1, :, 64:128].double() - want[:, 64:128]).abs() <= bound[:, 64:128] + 2.0 ** -24 * want[:, 64:128]).all()


# ---------------------------------------------------------------- selection
def check_select(w, lens, budget, sink, recent):
    B, heads, width = w.shape
    keep, counts, kept = binding.cache_select(w, ints(lens), budget, sink=sink, recent=recent)
    assert counts.tolist() == [min(n, budget) for n in lens]
    rows, mine = w.cpu(), kept.cpu()
    for b, n in enumerate(lens):
        c = min(n, budget)
        for h in range(heads):
            want = evict_util.select(rows[b, h].tolist(), n, budget, sink, recent)
            assert keep[b, h].tolist() == want + [-1] * (budget - c), (b, h)
            assert torch.equal(mine[b, h, :c].view(torch.int32), rows[b, h, want].view(torch.int32))
    live = torch.arange(width) < counts.cpu()[:, None, None]
    assert not mine.masked_fill(live, 0.0).any()


@pytest.mark.parametrize("B,heads,width,budget,sink,recent", [
    (1, 1, 1, 1, 0, 0), (1, 1, 40, 1, 0, 0), (2, 3, 31, 7, 1, 1), (3, 2, 1000, 256, 4, 32), (2, 2, 513, 512, 512, 0),
    (2, 2, 700, 600, 0, 600), (1, 8, 4097, 100, 50, 50), (4, 2, 9000, 4096, 3, 64), (70, 5, 600, 64, 2, 8),
    (2, 1, 20000, 19999, 7, 9), (1, 2, 33000, 1000, 0, 0), (1, 1, 131071, 16384, 16, 1024), (200, 2, 5000, 300, 0, 20),
    (1, 2, 150000, 20000, 9, 100), (160, 1, 19000, 5000, 3, 7), (3, 1, 2049, 2048, 0, 0), (2, 8, 70000, 69000, 33000, 33000)])
@pytest.mark.parametrize("kind", ["spread", "ties", "zeros"])
def test_select(B, heads, width, budget, sink, recent, kind):
    g = generator(width + budget)
    w = (torch.randn(B, heads, width, generator=g, device="cuda") * 2).exp()
    if kind == "ties":
        w = (w * 4).round().clamp(max=6) / 4
    elif kind == "zeros":
        w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.97, 0.0, w)
    rng = random.Random(width)
    lens = [width] + [rng.randint(0, width) for _ in range(B - 1)]
    check_select(w, lens, budget, sink, recent)


def test_select_rows_that_shared_memory_does_not_hold():
    g = generator(1)
    w = (torch.randn(2, 1, 500001, generator=g, device="cuda") * 2).exp()
    check_select(w, [500001, 400000], 30000, 5, 100)


@pytest.mark.parametrize("width,budget", [(60, 9), (5000, 700)])
def test_select_any_values(width, budget):
    """Signs, infinities, subnormals, -0 beside 0, and NaN, of any bits."""
    g = generator(width)
    bits = torch.randint(-1 << 31, 1 << 31, (4, 2, width), generator=g, device="cuda").to(torch.int32)
    w = bits.view(torch.float32).clone()
    some = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-40, -1e-40], device="cuda")
    w[1] = some[torch.randint(0, 7, (2, width), generator=g, device="cuda")]
    w[2] = some[torch.randint(0, 2, (2, width), generator=g, device="cuda")]
    w[3] = some[torch.randint(2, 5, (2, width), generator=g, device="cuda")]
    check_select(w, [width] * 4, budget, 2, 3)


def test_select_lengths_out_of_range_are_recorded():
    w = torch.rand(2, 1, 50, device="cuda")
    for bad in ([-1, 3], [10, 51]):
        _, counts, _ = binding.cache_select(w, ints(bad), 20)
        assert counts.tolist() == [min(max(n, 0), 20) for n in bad]
        assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN


# ---------------------------------------------------------------- moving
def moved(cache, lists, first, to_table, Hkv):
    """What the pages hold after the move."""
    k, v = cache.k.clone(), cache.v.clone()
    S = cache.page
    for b, heads in enumerate(lists):
        for h in range(Hkv):
            mine = heads[h if len(heads) > 1 else 0]
            if not mine:
                continue
            src = torch.tensor(mine, device="cuda")
            dst = torch.arange(len(mine), device="cuda") + first[b]
            a, z = cache.table[b].long()[src // S], to_table[b].long()[dst // S]
            k[z, h, dst % S] = cache.k[a, h, src % S]
            v[z, h, dst % S] = cache.v[a, h, src % S]
    return k, v


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


MOVES = [  # lens, counts, kv heads, d, page, dtype, slots first, one list for all heads
    ([40], [7], 2, 64, 16, torch.float16, False, False),
    ([1, 0, 16, 33], [1, 0, 16, 20], 3, 128, 16, torch.bfloat16, True, True),
    ([3000, 128, 129, 700], [2000, 64, 129, 0], 8, 128, 64, torch.bfloat16, False, False),
    ([5000, 2], [1234, 1], 2, 64, 256, torch.float16, False, False),
    ([900] * 30, [500] * 30, 4, 128, 32, torch.bfloat16, True, False),
    ([20000], [19000], 1, 128, 128, torch.float16, False, True),
    ([260] * 100, [6] * 100, 8, 128, 64, torch.bfloat16, False, True),
]


@pytest.mark.parametrize("move", MOVES, ids=lambda m: f"{str(m[0])[:16]}-{str(m[1])[:16]}-{m[2]}x{m[3]}")
@pytest.mark.parametrize("where", ["in place", "behind", "elsewhere"])
def test_keep(move, where):
    lens, counts, Hkv, d, page, dtype, slots_first, shared = move
    rng = random.Random(len(lens) + sum(counts))
    cache = Cache(lens, Hkv, d, page, dtype, slots_first=slots_first, seed=3, spare=2 + sum(-(-(c + 9) // page) for c in counts))
    used = {int(x) for x in cache.table.flatten() if x >= 0}
    free = [x for x in range(cache.k.shape[0]) if x not in used]
    first = [0] * len(lens)
    table, out_table = cache.table, None
    if where == "behind":  # a path among the last tokens
        counts = [min(c, (n + 1) // 2) for c, n in zip(counts, lens)]
        first = [rng.randint(0, n - c) for c, n in zip(counts, lens)]
    elif where == "elsewhere":
        first = [rng.randint(0, 9) for _ in lens]
        cols = max(-(-(c + f) // page) for c, f in zip(counts, first)) + 1
        rows = []
        for c, f in zip(counts, first):
            need = -(-(c + f) // page)
            rows.append([free.pop(rng.randrange(len(free))) for _ in range(need)] + [-3] * (cols - need))
        table = out_table = ints(rows)
    lists = []
    for b, (c, n) in enumerate(zip(counts, lens)):
        pick = (lambda: sorted(rng.sample(range(first[b], n), c))) if where != "elsewhere" else \
            (lambda: [rng.randrange(n) for _ in range(c)] if n else [])
        lists.append([pick() for _ in range(1 if shared else Hkv)])
    N = max(counts) + 3
    keep = ints([[x + [rng.randint(-9, 1 << 30) for _ in range(N - len(x))] for x in heads] for heads in lists])
    want = moved(cache, lists, first, table, Hkv)
    pages = binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, keep, ints([len(x[0]) for x in lists]),
                               first=None if where == "in place" else ints(first), out_table=out_table)
    assert pages[0] is cache.k and pages[1] is cache.v
    assert same_bits(cache.k, want[0]) and same_bits(cache.v, want[1])


def test_keep_faults_are_recorded_and_passed_over():
    lens = [100, 60]
    cache = Cache(lens, 2, 64, 16, torch.float16, seed=2)
    keep = torch.zeros(2, 1, 5, dtype=torch.int32, device="cuda")
    for rows, counts, first, status in (
            ([[0, 5, 1, 7, 8]] * 2, [5, 2], [0, 0], binding.FA_ERR_INDEX),    # 1 stands in front of its place
            ([[3, 5, 100, 107, 50]] * 2, [5, 2], [0, 0], binding.FA_ERR_INDEX),
            ([[-1, 5, 6, 7, 8]] * 2, [5, 2], [0, 0], binding.FA_ERR_INDEX),
            ([[1, 2, 3, 4, 5]] * 2, [6, 1], [0, 0], binding.FA_ERR_SEQ_LEN),
            ([[1, 2, 3, 4, 5]] * 2, [5, -1], [0, 0], binding.FA_ERR_SEQ_LEN),
            ([[1, 2, 3, 4, 5]] * 2, [5, 1], [-1, 0], binding.FA_ERR_SEQ_LEN)):
        keep[:, 0] = ints(rows)
        a, n = max(first[0], 0), min(max(counts[0], 0), 5)
        k, v = cache.k.clone(), cache.v.clone()
        for b in range(2):
            src0, S = rows[b], 16
            take = [(s, max(first[b], 0) + i) for i, s in enumerate(src0[:min(max(counts[b], 0), 5)])]
            for s, t in take:
                if s < t or s >= lens[b]:
                    continue
                for x, y in ((k, cache.k), (v, cache.v)):
                    x[int(cache.table[b, t // S]), :, t % S] = y[int(cache.table[b, s // S]), :, s % S]
        binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, keep, ints(counts), first=ints(first))
        assert binding.fa_device_status(True) == status, (rows, counts, first)
        assert same_bits(cache.k, k) and same_bits(cache.v, v)
    # a new page outside the cache is not written, tokens of an old one move as zeros
    keep[:, 0] = ints([[0, 1, 2, 3, 4]] * 2)
    out = ints([[cache.k.shape[0]], [-1]])
    k, v = cache.k.clone(), cache.v.clone()
    binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, keep, ints([5, 5]), out_table=out)
    assert binding.fa_device_status(True) == binding.FA_ERR_PAGE
    assert same_bits(cache.k, k) and same_bits(cache.v, v)
    bad, spare = cache.table.clone(), [x for x in range(cache.k.shape[0]) if x not in cache.table.flatten().tolist()]
    bad[0, 0] = -5
    binding.cache_keep(cache.k, cache.v, bad, cache.seq_lens, keep, ints([5, 5]), out_table=ints([[spare[0]], [spare[1]]]))
    assert binding.fa_device_status(True) == binding.FA_ERR_PAGE
    assert not cache.k[spare[0], :, :5].any() and not cache.v[spare[0], :, :5].any()
    assert same_bits(cache.k[spare[1], :, :5], cache.k[int(cache.table[1, 0]), :, :5])


def test_keep_far_pages():
    cache = Cache([300], 2, 128, 64, torch.float16, total_pages=(1 << 32) // (2 * 128 * 64) + 9, behind=0.0)
    keys, values = cache.keys(0)
    mine = sorted(random.Random(1).sample(range(300), 150))
    binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, ints([[mine]]), ints([150]))
    for x, y in ((cache.k, keys), (cache.v, values)):
        got = x[cache.table[0, :3].long()].transpose(1, 2).reshape(-1, 2, 128)[:150].double()
        assert torch.equal(got, y[mine])


# ---------------------------------------------------------------- together
def test_a_captured_eviction_follows_lengths_that_change():
    """Weigh, select and keep in one graph on a stream of its own, replayed on other lengths, against the eager calls."""
    lens, Hq, Hkv, d, page, budget = [900, 500, 1200], 8, 2, 64, 32, 300
    side = torch.cuda.Stream()
    one, two = (Cache(lens, Hkv, d, page, torch.float16, seed=4) for _ in range(2))
    q = torch.randn(3, Hq, d, generator=generator(6), device="cuda").half()
    lse = torch.full((3, Hq), 6.0, device="cuda")
    w = torch.rand(3, Hkv, 1300, generator=generator(7), device="cuda")
    wide = torch.zeros_like(w)
    torch.cuda.synchronize()

    def step(cache, out):
        binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, weights=w, decay=0.5, out=out)
        keep, counts, kept = binding.cache_select(out, cache.seq_lens, budget, sink=4, recent=16)
        binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, keep, counts)
        return keep, counts, kept

    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(one, wide)
    for now in (lens, [301, 200, 1100], [300, 0, 299]):
        for c in (one, two):
            c.seq_lens.copy_(ints(now))
        wide.zero_()
        want = step(two, torch.zeros_like(w))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert same_bits(one.k, two.k) and same_bits(one.v, two.v)


def test_drafts_checked_and_kept():
    """A serving step with drafted trees: append the nodes, check them in one pass, keep a path, go on with the next token."""
    Hq, Hkv, d, page, dtype = 8, 2, 64, 16, torch.float16
    had, counts = [100, 37, 15], [12, 7, 20]
    rng = random.Random(8)
    cols = 10
    pages = [torch.full((3 * cols, Hkv, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
    table = torch.randperm(3 * cols, generator=generator(1), device="cuda").to(torch.int32).view(3, cols)
    rope = binding.rope_table(400, d)
    g = generator(2)
    # the context: raw keys turned at their positions
    ctx = [torch.randn(2, n, Hkv, d, generator=g, device="cuda").to(dtype) for n in had]
    lens = ints(had)
    binding.cache_append(None, *(torch.cat([c[i] for c in ctx]) for i in range(2)), *pages, table, lens, ints(offsets(had)), rope)
    # the trees
    trees = [[rng.randint(max(-1, i - 4), i - 1) for i in range(n)] for n in counts]
    new = torch.randn(sum(counts), Hq + 2 * Hkv, d, generator=g, device="cuda").to(dtype)
    q, k, v = new[:, :Hq], new[:, Hq:Hq + Hkv], new[:, Hq + Hkv:]
    cu = ints(offsets(counts))
    lens += ints(counts)
    mask, positions = binding.tree_mask(ints(sum(trees, [])), cu, max(counts), lens)
    turned = binding.cache_append(q, k, v, *pages, table, lens, cu, rope, positions=positions)
    out = binding.prefill_tree(turned, *pages, table, lens, cu, max(counts), mask)
    # every node's path as a sequence of its own
    paths = []
    for b, tree in enumerate(trees):
        paths.append([])
        for i in range(counts[b]):
            path = [i]
            while tree[path[0]] >= 0:
                path.insert(0, tree[path[0]])
            paths[b].append(path)
    t = 0
    for b, n in enumerate(counts):
        for i in (0, n // 2, n - 1):
            path = paths[b][i]
            plain = [torch.zeros(cols, Hkv, page, d, dtype=dtype, device="cuda") for _ in range(2)]
            length, t1 = had[b] + len(path), ints(list(range(cols)))[None]
            binding.cache_append(None, *(torch.cat([ctx[b][j], x[[t + p for p in path]]]) for j, x in ((0, k), (1, v))), *plain, t1,
                                 ints([length]), ints([0, length]), rope)
            want = binding.decode_paged(turned[t + i][None].contiguous(), *plain, t1, ints([length]))
            # both round weights to fp16 and sum in fp32, in orders of their own: twice a value's bound of 2^-11 (|o| and the mean |v|)
            spread = torch.cat([ctx[b][1], v[[t + p for p in path]]]).double().abs().amax()
            assert ((out[t + i].double() - want[0].double()).abs() <= 4 * 2.0 ** -11 * spread).all()
        t += n
    # keep a longest path, and decode behind it
    best = [max(p, key=len) for p in paths]
    took = [len(p) for p in best]
    base = lens - ints(counts)
    keep = ints([[[n + i for i in p] + [-1] * (max(took) - len(p))] for n, p in zip(had, best)])
    binding.cache_keep(*pages, table, lens, keep, ints(took), first=base)
    lens = base + ints(took)
    nxt = torch.randn(3, Hq, d, generator=g, device="cuda").to(dtype)
    got = binding.decode_paged(nxt, *pages, table, lens)
    for b in range(3):
        rows = [sum(counts[:b]) + i for i in best[b]]
        plain = [torch.zeros(cols, Hkv, page, d, dtype=dtype, device="cuda") for _ in range(2)]
        t1, length = ints(list(range(cols)))[None], had[b] + took[b]
        binding.cache_append(None, *(torch.cat([ctx[b][j], x[rows]]) for j, x in ((0, k), (1, v))), *plain, t1, ints([length]),
                             ints([0, length]), rope)
        for x, y in zip(pages, plain):
            mine = x[table[b].long()].transpose(1, 2).reshape(-1, Hkv, d)[:length]
            assert torch.equal(mine, y.transpose(1, 2).reshape(-1, Hkv, d)[:length])
        want = binding.decode_paged(nxt[b:b + 1], *plain, t1, ints([length]))
        spread = max(ctx[b][1].abs().max(), v[rows].abs().max()).double()
        assert ((got[b].double() - want[0].double()).abs() <= 4 * 2.0 ** -11 * spread).all()


def test_a_cache_kept_at_a_budget():
    """Prefill, weigh, select, keep, then decode with appended tokens: the same rows as attention over the kept tokens."""
    Hq, Hkv, d, page, dtype, budget = 8, 2, 128, 64, torch.bfloat16, 256
    lens = [700, 150, 1000]
    cache = Cache(lens, Hkv, d, page, dtype, seed=9, extra_cols=3)
    raw = [tuple(x.clone() for x in cache.keys(b)) for b in range(3)]
    q = torch.randn(sum(lens), Hq, d, generator=generator(3), device="cuda").to(dtype)
    cu, lse = ints(offsets(lens)), torch.empty(sum(lens), Hq, device="cuda")
    binding.prefill_paged(q, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(lens), causal=True, lse=lse)
    width = cache.table.shape[1] * page
    w = binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(lens))
    assert w.shape[2] == width
    keep, counts, w = binding.cache_select(w, cache.seq_lens, budget, sink=4, recent=32)
    binding.cache_keep(cache.k, cache.v, cache.table, cache.seq_lens, keep, counts)
    now = counts + 1
    new = torch.randn(3, Hq + 2 * Hkv, d, generator=generator(4), device="cuda").to(dtype)
    rope = binding.rope_table(1100, d)
    turned = binding.cache_append(new[:, :Hq], new[:, Hq:Hq + Hkv], new[:, Hq + Hkv:], cache.k, cache.v, cache.table, now, rope=rope,
                                  positions=ints(lens))
    one = torch.empty(3, Hq, device="cuda")
    out = torch.empty_like(turned)
    binding.prefill_paged(turned, cache.k, cache.v, cache.table, now, ints([0, 1, 2, 3]), 1, lse=one, out=out)
    binding.cache_weigh(turned, one, cache.k, cache.v, cache.table, now, weights=w, out=w)
    for b in range(3):
        n = min(lens[b], budget)
        place = (int(cache.table[b, n // page]), slice(None), n % page)
        for h in range(Hkv):
            mine = keep[b, h, :n].long()
            k = torch.cat([raw[b][0][mine, h], cache.k[place][h].double()[None]])[:, None]
            v = torch.cat([raw[b][1][mine, h], cache.v[place][h].double()[None]])[:, None]
            rows = turned[b:b + 1, h * 4:h * 4 + 4].double()
            seen = torch.ones(1, n + 1, dtype=torch.bool, device="cuda")
            want, _, bound, off = evict_util.attend_seen(rows, k, v, 1 / math.sqrt(d), seen, dtype)
            err = (out[b:b + 1, h * 4:h * 4 + 4].double() - want).abs()
            assert (err <= bound + 2.0 ** -8 * (want.abs() + bound)).all()
            # the new token's own weight came on a zero, and all of them were added to
            p, tol = evict_util.weigh(rows, k, one[b:b + 1, h * 4:h * 4 + 4].double(), 1 / math.sqrt(d), seen)
            assert ((w[b, h, n].double() - p[0, n]).abs() <= tol[0, n] + 2.0 ** -24 * p[0, n]).all()
            assert not w[b, h, n + 1:].any()


def test_two_streams_at_once():
    """The same calls on two streams at a time come out as one after the other."""
    forms = [FORMS[6], FORMS[1]]
    made = [run_weigh(f) for f in forms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in forms]
    again = []
    for _ in range(5):
        for s, f, (cache, q, lse, cu, news, w, out) in zip(streams, forms, made):
            with torch.cuda.stream(s):
                got = torch.full_like(out, 7.0)
                binding.cache_weigh(q, lse, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(news), weights=w, decay=0.75, out=got)
                again.append((got, out, binding.cache_select(out, cache.seq_lens, 60, recent=5)))
    torch.cuda.synchronize()
    for i, (got, out, sel) in enumerate(again):
        assert torch.equal(got, out)
        assert all(torch.equal(a, b) for a, b in zip(sel, again[i % 2][2]))
