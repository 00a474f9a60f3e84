"""Drafted trees on the GPU: masks and positions against walks up the trees, attention under masks against the definition
in 64 bits over all three kernels, calls in CUDA graphs and on other streams, faults on the device."""
import math
import random

import pytest
import torch

from attention_forward_prefill_gb300 import binding
from tests.evict_util import attend_seen, mask_of, seen_of
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


def some_tree(rng, n, spread):
    return [rng.randint(max(-1, i - spread), i - 1) for i in range(n)]


@pytest.mark.parametrize("counts,spread", [([1], 1), ([8], 3), ([0, 1, 31, 0, 32, 33, 0], 5), ([64, 65, 127, 128, 129], 40),
                                           ([300, 2, 257], 1), ([4096, 1], 1000), ([4097, 5000], 700), ([1100], 1), ([7] * 300, 2)])
def test_mask(counts, spread):
    rng = random.Random(sum(counts) + spread)
    trees = [some_tree(rng, n, spread) for n in counts]
    lens = [n + rng.randint(0, 9) for n in counts]
    most = max(counts)
    mask, pos = binding.tree_mask(ints(sum(trees, [])), ints(offsets(counts)), most, ints(lens))
    want, at = [], []
    for t, n in zip(trees, lens):
        rows, depth = mask_of(t, -(-most // 32))
        want += rows
        at += [n - len(t) + x for x in depth]
    assert torch.equal(mask.cpu(), torch.tensor(want, dtype=torch.int32))
    assert torch.equal(pos.cpu(), torch.tensor(at, dtype=torch.int32))
    mask2, none = binding.tree_mask(ints(sum(trees, [])), ints(offsets(counts)), most + 40)
    assert none is None and torch.equal(mask2[:, :mask.shape[1]], mask) and not mask2[:, mask.shape[1]:].any()


def test_mask_rows_outside_sequences_stay():
    words = torch.full((10, 1), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((10,), 78, dtype=torch.int32, device="cuda")
    parents, cu, lens = ints([-1] * 10), ints([2, 4, 7]), ints([5, 6])
    stream = torch.cuda.current_stream().cuda_stream
    assert binding.fa_tree_mask(parents.data_ptr(), words.data_ptr(), 1, pos.data_ptr(), lens.data_ptr(), cu.data_ptr(), 2, 10, 8,
                                stream) == 0
    assert words[:, 0].tolist() == [77, 77, 1, 2, 1, 2, 4, 77, 77, 77]
    assert pos.tolist() == [78, 78, 3, 3, 3, 3, 3, 78, 78, 78]


@pytest.mark.parametrize("parents,like", [([-1, 1, 0], [-1, -1, 0]), ([-1, 0, -2], [-1, 0, -1]), ([5, 0, 2], [-1, 0, -1]),
                                          ([-1, 0, 1 << 30], [-1, 0, -1])])
def test_mask_bad_parents_are_recorded(parents, like):
    mask, pos = binding.tree_mask(ints(parents), ints([0, 3]), 3, ints([3]))
    assert binding.fa_device_status(True) == binding.FA_ERR_INDEX
    rows, depth = mask_of(like, 1)
    assert mask.cpu().tolist() == rows and pos.tolist() == depth


def test_mask_bad_offsets_are_recorded():
    for cu in ([0, 5], [-1, 3], [0, 1 << 30]):
        binding.tree_mask(ints([-1] * 4), ints(cu), 4, ints([9]))
        assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN
    binding.tree_mask(ints([-1] * 4), ints([0, 4]), 3)
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN


# (lens, query tokens, query heads, kv heads, d, page, dtype, slots first): few and many rows per kv head, short and long tables
FORMS = [
    ([1000], [12], 12, 12, 64, 16, torch.float16, False),            # 12 rows: a cluster
    ([1], [1], 4, 2, 128, 16, torch.bfloat16, False),
    ([5, 64, 65], [5, 64, 65], 2, 2, 64, 32, torch.bfloat16, True),  # no context at all
    ([3, 0, 70], [9, 4, 70], 4, 1, 128, 64, torch.float16, False),   # more query tokens than keys
    ([700, 40, 2000], [8, 0, 3], 32, 8, 128, 64, torch.bfloat16, False),
    ([700, 64, 300], [16, 7, 10], 14, 7, 64, 16, torch.float16, True),
    ([9000, 300, 5000], [8, 5, 8], 16, 2, 128, 128, torch.bfloat16, False),    # 64 rows over long tables: ranges
    ([20000, 1, 130], [4, 1, 2], 16, 4, 64, 64, torch.float16, False),         # 16 rows
    ([9000, 3000], [7, 5], 16, 4, 128, 256, torch.float16, True),              # 28 rows
    ([1500, 90, 128], [33, 64, 17], 32, 8, 128, 64, torch.bfloat16, False),    # over 64 rows: tensor-memory tiles
    ([4000, 333], [100, 130], 14, 2, 64, 16, torch.float16, True),
    ([260, 129, 128], [260, 127, 128], 6, 2, 128, 32, torch.float16, False),
    ([600, 257], [300, 1], 5, 5, 64, 64, torch.bfloat16, False),
    ([300], [80], 130, 1, 64, 64, torch.float16, False),                       # a group over 128
]


def run_tree(form, make_mask, seed=0, **more):
    lens, counts, Hq, Hkv, d, page, dtype, slots_first = form
    cache = Cache(lens, Hkv, d, page, dtype, slots_first=slots_first, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn(sum(counts), Hq, d, generator=g, device="cuda") * 1.5).to(dtype)
    mask = make_mask(counts)
    lse = torch.empty(sum(counts), Hq, device="cuda")
    out = binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts)), max(counts), mask, lse=lse,
                               **more)
    return cache, q, mask, lse, out


def check_tree(form, cache, q, mask, lse, out, scale):
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    t = 0
    for b, n in enumerate(counts):
        if n == 0:
            continue
        k, v = cache.keys(b)
        seen = seen_of(mask[t:t + n], n, lens[b])
        want, want_lse, bound, off = attend_seen(q[t:t + n].double(), k, v, scale, seen, dtype)
        assert_rows(out[t:t + n], want, bound, f"sequence {b}")
        none = want_lse == -math.inf
        assert torch.equal(lse[t:t + n] == -math.inf, none)
        assert ((lse[t:t + n].double() - want_lse)[~none].abs() <= off[~none]).all()
        t += n


def trees_mask(counts, spread=6, seed=3):
    rng = random.Random(seed)
    words = -(-max(counts) // 32)
    return ints(sum((mask_of(some_tree(rng, n, spread), words)[0] for n in counts), []))


def any_mask(counts):
    """Bits as they come, those of tokens that there are not among them, and some rows without any."""
    g = torch.Generator(device="cuda").manual_seed(9)
    words = -(-max(counts) // 32)
    m = torch.randint(-1 << 31, 1 << 31, (sum(counts), words), generator=g, device="cuda").to(torch.int32)
    m[torch.rand(m.shape[0], generator=g, device="cuda") < 0.3] = 0
    return m


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f[0]}-{f[1]}-{f[2]}over{f[3]}x{f[4]}")
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_tree(form, kind):
    scale = 1 / math.sqrt(form[4])
    args = run_tree(form, trees_mask if kind == "tree" else any_mask)
    check_tree(form, *args, scale)


@pytest.mark.parametrize("form", [FORMS[4], FORMS[6], FORMS[9]], ids=["cluster", "ranges", "tiles"])
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_tree_scales(form, scale):
    check_tree(form, *run_tree(form, any_mask, scale=scale, out_dtype=torch.float32), scale)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: f"{f[0]}-{f[1]}-{f[2]}over{f[3]}x{f[4]}")
def test_a_chain_is_causal(form):
    """A tree in which every node follows the one before is what prefill_paged computes causally."""
    lens, counts = form[0], form[1]
    chain = lambda c: ints(sum((mask_of(list(range(-1, n - 1)), -(-max(c) // 32))[0] for n in c), []))  # noqa: E731
    cache, q, mask, lse, out = run_tree(form, chain, out_dtype=torch.float32)
    want = binding.prefill_paged(q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts)), max(counts), causal=True,
                                 out_dtype=torch.float32)
    t = 0
    for b, n in enumerate(counts):
        if n:
            bound = attend_seen(q[t:t + n].double(), *cache.keys(b), 1 / math.sqrt(form[4]), seen_of(mask[t:t + n], n, lens[b]), form[6])[2]
            # each is within the bound of the definition, and rounds once to fp32
            assert ((out - want)[t:t + n].double().abs() <= 2 * bound + 2.0 ** -23 * want[t:t + n].abs()).all()
        t += n


@pytest.mark.parametrize("form", [FORMS[4], FORMS[6], FORMS[9]], ids=["cluster", "ranges", "tiles"])
def test_hidden_keys_may_be_nan(form):
    """What no bit shows takes no part: NaN and infinities among the keys of nodes that nobody sees."""
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    cache, q, mask, lse, out = run_tree(form, lambda c: trees_mask(c) & 0x15555555)
    for value in (math.nan, math.inf, -math.inf):
        for b, n in enumerate(counts):
            for j in range(1, n, 2):
                at = lens[b] - n + j
                cache.k[int(cache.table[b, at // page]), :, at % page] = value
        again = binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts)), max(counts), mask)
        assert torch.equal(again, out)


@pytest.mark.parametrize("form", [FORMS[4], FORMS[6], FORMS[9]], ids=["cluster", "ranges", "tiles"])
def test_runs_alike_with_a_workspace_and_leaves_other_rows(form):
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    cache, q, mask, lse, out = run_tree(form, any_mask)
    total = sum(counts)
    wide_q = torch.cat([torch.full((2, Hq, d), math.nan, dtype=dtype, device="cuda"), q, q[:3]])
    wide_mask = torch.cat([mask[:2], mask, mask[:3]])
    wide_out = torch.full((total + 5, Hq, d), 7.0, dtype=dtype, device="cuda")
    ws = torch.empty(binding.fa_paged_workspace_bytes(Hq, Hkv, max(counts), d) + 16, dtype=torch.uint8, device="cuda")
    binding.prefill_tree(wide_q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts, 2)), max(counts), wide_mask,
                         workspace=ws, out=wide_out)
    assert torch.equal(wide_out[2:2 + total], out)
    assert (wide_out[:2] == 7).all() and (wide_out[2 + total:] == 7).all()
    with pytest.raises(binding.FaError, match="WORKSPACE"):
        binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts)), max(counts), mask, workspace=ws[:64])


def test_a_captured_call_follows_what_it_reads():
    lens, counts, Hq, Hkv, d, page, dtype, _ = form = FORMS[9]
    side = torch.cuda.Stream()
    cache, q, mask, lse, out = run_tree(form, any_mask)
    cu, parents = ints(offsets(counts)), ints(sum((some_tree(random.Random(1), n, 5) for n in counts), []))
    made = torch.empty_like(out)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        binding.tree_mask(parents, cu, max(counts), cache.seq_lens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            bits, pos = binding.tree_mask(parents, cu, max(counts), cache.seq_lens)
            binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, cu, max(counts), bits, out=made)
    for seed, shorter in ((2, 0), (3, 5)):
        trees = [some_tree(random.Random(seed + n), n, 4) for n in counts]
        parents.copy_(ints(sum(trees, [])))
        now = [n - shorter for n in lens]
        cache.seq_lens.copy_(ints(now))
        graph.replay()
        torch.cuda.synchronize()
        t = 0
        for b, n in enumerate(counts):
            k, v = cache.keys(b)
            rows = torch.tensor(mask_of(trees[b], bits.shape[1])[0], dtype=torch.int32, device="cuda")
            assert torch.equal(bits[t:t + n], rows)
            want, _, bound, _ = attend_seen(q[t:t + n].double(), k[:now[b]], v[:now[b]], 1 / math.sqrt(d), seen_of(rows, n, now[b]), dtype)
            assert_rows(made[t:t + n], want, bound, f"replay {seed}, sequence {b}")
            t += n


def test_far_pages_and_bad_pages():
    """Pages behind 2^32 elements, a page that is none, and a length that is too long."""
    form = ([300, 140], [20, 70], 4, 2, 128, 64, torch.float16, False)
    lens, counts, Hq, Hkv, d, page, dtype, _ = form
    cache = Cache(lens, Hkv, d, page, dtype, total_pages=(1 << 32) // (Hkv * d * page) + 9, behind=0.0)
    q = torch.randn(sum(counts), Hq, d, device="cuda").to(dtype)
    mask, lse = any_mask(counts), torch.empty(sum(counts), Hq, device="cuda")
    out = binding.prefill_tree(q, cache.k, cache.v, cache.table, cache.seq_lens, ints(offsets(counts)), max(counts), mask, lse=lse)
    check_tree(form, cache, q, mask, lse, out, 1 / math.sqrt(d))
    bad = cache.table.clone()
    bad[0, 1] = cache.k.shape[0]
    binding.prefill_tree(q, cache.k, cache.v, bad, cache.seq_lens, ints(offsets(counts)), max(counts), mask)
    assert binding.fa_device_status(True) == binding.FA_ERR_PAGE
    wide = torch.cat([cache.table[:, :1]] * 5, 1)
    binding.prefill_tree(q, cache.k, cache.v, wide.contiguous(), ints([321, 140]), ints(offsets(counts)), max(counts), mask)
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN
