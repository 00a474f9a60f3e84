"""Drafted trees and eviction without a GPU: bad arguments come back as the documented status before any CUDA call."""
import pytest

from attention_forward_prefill_gb300 import binding, build
from tests.test_paged_host import CACHE_REFUSALS, cache

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()


def pick(defaults, change):
    return [change.get(k, v) for k, v in defaults.items()]


def mask(**c):
    return binding.fa_tree_mask(*pick(dict(parents=1 << 32, mask=2 << 32, words=2, positions=3 << 32, lens=4 << 32, cu=5 << 32, B=4,
                                           total=100, most=64), c))


@pytest.mark.parametrize("change,status", [
    (dict(parents=None), binding.FA_ERR_NULL), (dict(mask=None), binding.FA_ERR_NULL), (dict(cu=None), binding.FA_ERR_NULL),
    (dict(lens=None), binding.FA_ERR_NULL), (dict(B=0), binding.FA_ERR_SHAPE), (dict(total=-1), binding.FA_ERR_SHAPE),
    (dict(most=0), binding.FA_ERR_SHAPE), (dict(words=0), binding.FA_ERR_SHAPE), (dict(most=65), binding.FA_ERR_SHAPE),
    (dict(total=1 << 30), binding.FA_ERR_SHAPE), (dict(most=1 << 20, words=1 << 15, B=1 << 20), binding.FA_ERR_SHAPE),
    (dict(parents=(1 << 32) + 2), binding.FA_ERR_ALIGN), (dict(mask=(2 << 32) + 1), binding.FA_ERR_ALIGN),
    (dict(positions=(3 << 32) + 2), binding.FA_ERR_ALIGN), (dict(lens=(4 << 32) + 2), binding.FA_ERR_ALIGN),
    (dict(cu=(5 << 32) + 2), binding.FA_ERR_ALIGN), (dict(mask=1 << 32), binding.FA_ERR_ALIAS),
    (dict(mask=(1 << 32) - 796), binding.FA_ERR_ALIAS), (dict(positions=(1 << 32) + 396), binding.FA_ERR_ALIAS),
    (dict(positions=2 << 32), binding.FA_ERR_ALIAS), (dict(positions=(4 << 32) + 12), binding.FA_ERR_ALIAS),
    (dict(mask=(5 << 32) + 16), binding.FA_ERR_ALIAS)])
def test_mask_refusals(change, status):
    assert mask(**change) == status


def tree(**c):
    a = pick(dict(q=3 << 32, out=6 << 32, lse=12 << 32, page_table=7 << 32, max_pages=10, seq_lens=8 << 32, cu=9 << 32, mask=10 << 32,
                  words=1, B=4, Hq=32, total=9, max_q=5, scale=0.1, out_dtype=binding.FA_BF16, ws=None, ws_bytes=0), c)
    return binding.fa_prefill_tree(cache(**c), *a)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(q=None), binding.FA_ERR_NULL), (dict(out=None), binding.FA_ERR_NULL), (dict(page_table=None), binding.FA_ERR_NULL),
    (dict(seq_lens=None), binding.FA_ERR_NULL), (dict(cu=None), binding.FA_ERR_NULL), (dict(mask=None), binding.FA_ERR_NULL),
    (dict(words=0), binding.FA_ERR_SHAPE), (dict(max_q=33), binding.FA_ERR_SHAPE), (dict(B=0), binding.FA_ERR_SHAPE),
    (dict(Hq=33), binding.FA_ERR_SHAPE), (dict(max_q=0), binding.FA_ERR_SHAPE), (dict(total=-1), binding.FA_ERR_SHAPE),
    (dict(out_dtype=7), binding.FA_ERR_DTYPE), (dict(mask=(10 << 32) + 2), binding.FA_ERR_ALIGN), (dict(lse=(12 << 32) + 2), binding.FA_ERR_ALIGN),
    (dict(scale=INF), binding.FA_ERR_SCALE), (dict(out=10 << 32), binding.FA_ERR_ALIAS), (dict(lse=(10 << 32) + 32), binding.FA_ERR_ALIAS),
    (dict(out=3 << 32), binding.FA_ERR_ALIAS), (dict(lse=6 << 32), binding.FA_ERR_ALIAS)])
def test_tree_refusals(change, status):
    assert tree(**change) == status


def weigh(**c):
    a = pick(dict(q=3 << 32, lse=12 << 32, page_table=7 << 32, max_pages=10, seq_lens=8 << 32, cu=9 << 32, B=4, Hq=32, total=9, max_q=5,
                  causal=1, scale=0.1, weights=6 << 32, decay=0.9, out=6 << 32, width=640), c)
    return binding.fa_cache_weigh(cache(**c), *a)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(q=None), binding.FA_ERR_NULL), (dict(lse=None), binding.FA_ERR_NULL), (dict(page_table=None), binding.FA_ERR_NULL),
    (dict(seq_lens=None), binding.FA_ERR_NULL), (dict(out=None), binding.FA_ERR_NULL), (dict(B=0), binding.FA_ERR_SHAPE),
    (dict(Hq=33), binding.FA_ERR_SHAPE), (dict(max_pages=0), binding.FA_ERR_SHAPE), (dict(total=-1), binding.FA_ERR_SHAPE),
    (dict(total=1 << 27), binding.FA_ERR_SHAPE), (dict(max_q=0), binding.FA_ERR_SHAPE), (dict(width=0), binding.FA_ERR_SHAPE),
    (dict(width=1 << 30), binding.FA_ERR_SHAPE), (dict(cu=None), binding.FA_ERR_SHAPE), (dict(B=1 << 24, width=1 << 20), binding.FA_ERR_SHAPE),
    (dict(q=(3 << 32) + 8), binding.FA_ERR_ALIGN), (dict(lse=(12 << 32) + 2), binding.FA_ERR_ALIGN),
    (dict(weights=(6 << 32) + 2), binding.FA_ERR_ALIGN), (dict(out=(6 << 32) + 1), binding.FA_ERR_ALIGN),
    (dict(cu=(9 << 32) + 2), binding.FA_ERR_ALIGN), (dict(scale=NAN), binding.FA_ERR_SCALE), (dict(scale=3e38), binding.FA_ERR_SCALE),
    (dict(decay=NAN), binding.FA_ERR_SCALE), (dict(decay=INF), binding.FA_ERR_SCALE), (dict(out=(6 << 32) + 4), binding.FA_ERR_ALIAS),
    (dict(out=3 << 32), binding.FA_ERR_ALIAS), (dict(out=(12 << 32) + 1148), binding.FA_ERR_ALIAS), (dict(out=1 << 32), binding.FA_ERR_ALIAS),
    (dict(out=(7 << 32) + 156), binding.FA_ERR_ALIAS), (dict(out=(8 << 32) + 12), binding.FA_ERR_ALIAS), (dict(out=9 << 32), binding.FA_ERR_ALIAS)])
def test_weigh_refusals(change, status):
    assert weigh(**change) == status


def select(**c):
    return binding.fa_cache_select(*pick(dict(weights=1 << 32, lens=2 << 32, B=4, heads=8, width=1000, budget=100, sink=4, recent=20,
                                              keep=3 << 32, counts=4 << 32, kept=5 << 32), c))


@pytest.mark.parametrize("change,status", [
    (dict(weights=None), binding.FA_ERR_NULL), (dict(lens=None), binding.FA_ERR_NULL), (dict(keep=None), binding.FA_ERR_NULL),
    (dict(counts=None), binding.FA_ERR_NULL), (dict(B=0), binding.FA_ERR_SHAPE), (dict(heads=0), binding.FA_ERR_SHAPE),
    (dict(width=0), binding.FA_ERR_SHAPE), (dict(budget=0), binding.FA_ERR_SHAPE), (dict(sink=-1), binding.FA_ERR_SHAPE),
    (dict(recent=-1), binding.FA_ERR_SHAPE), (dict(sink=81), binding.FA_ERR_SHAPE), (dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1), binding.FA_ERR_SHAPE),
    (dict(width=1 << 30), binding.FA_ERR_SHAPE), (dict(budget=1 << 30), binding.FA_ERR_SHAPE), (dict(B=1 << 25), binding.FA_ERR_SHAPE),
    (dict(weights=(1 << 32) + 2), binding.FA_ERR_ALIGN), (dict(keep=(3 << 32) + 1), binding.FA_ERR_ALIGN),
    (dict(kept=(5 << 32) + 2), binding.FA_ERR_ALIGN), (dict(kept=1 << 32), binding.FA_ERR_ALIAS), (dict(keep=(1 << 32) + 127996), binding.FA_ERR_ALIAS),
    (dict(counts=(2 << 32) + 12), binding.FA_ERR_ALIAS), (dict(kept=3 << 32), binding.FA_ERR_ALIAS), (dict(counts=(5 << 32) + 8), binding.FA_ERR_ALIAS)])
def test_select_refusals(change, status):
    assert select(**change) == status


def keep(**c):
    a = pick(dict(page_table=7 << 32, max_pages=10, seq_lens=8 << 32, keep=9 << 32, heads=8, keep_len=50, counts=10 << 32, first=11 << 32,
                  out_table=None, out_pages=0, B=4), c)
    return binding.fa_cache_keep(cache(**c), *a)


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(page_table=None), binding.FA_ERR_NULL), (dict(seq_lens=None), binding.FA_ERR_NULL), (dict(keep=None), binding.FA_ERR_NULL),
    (dict(counts=None), binding.FA_ERR_NULL), (dict(B=0), binding.FA_ERR_SHAPE), (dict(max_pages=0), binding.FA_ERR_SHAPE),
    (dict(max_pages=1 << 25), binding.FA_ERR_SHAPE), (dict(heads=2), binding.FA_ERR_SHAPE), (dict(keep_len=0), binding.FA_ERR_SHAPE),
    (dict(keep_len=1 << 30), binding.FA_ERR_SHAPE), (dict(B=1 << 23), binding.FA_ERR_SHAPE), (dict(out_table=12 << 32), binding.FA_ERR_SHAPE),
    (dict(out_table=12 << 32, out_pages=1 << 25), binding.FA_ERR_SHAPE), (dict(out_table=7 << 32, out_pages=9), binding.FA_ERR_SHAPE),
    (dict(keep=(9 << 32) + 2), binding.FA_ERR_ALIGN), (dict(counts=(10 << 32) + 1), binding.FA_ERR_ALIGN),
    (dict(first=(11 << 32) + 2), binding.FA_ERR_ALIGN), (dict(out_table=(12 << 32) + 2, out_pages=3), binding.FA_ERR_ALIGN),
    (dict(keep=1 << 32), binding.FA_ERR_ALIAS), (dict(counts=(2 << 32) + 64), binding.FA_ERR_ALIAS),
    (dict(out_table=2 << 32, out_pages=3), binding.FA_ERR_ALIAS), (dict(v_pages=1 << 32), binding.FA_ERR_ALIAS)])
def test_keep_refusals(change, status):
    assert keep(**change) == status


def test_what_is_fine_reaches_the_device_check():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: only where no device can be reached")
    for rc in (mask(), mask(positions=None, lens=None), tree(), tree(lse=None), tree(max_q=32), weigh(), weigh(weights=None),
               weigh(weights=13 << 32), weigh(cu=None, total=20), select(), select(kept=None), select(sink=40, recent=60),
               keep(), keep(heads=1, first=None), keep(out_table=12 << 32, out_pages=3), keep(out_table=7 << 32, out_pages=10)):
        assert rc == binding.FA_ERR_CUDA


def test_status_text():
    assert binding.STATUS_NAMES[binding.FA_ERR_INDEX] == "FA_ERR_INDEX"
    assert "index" in binding.status_string(binding.FA_ERR_INDEX)


def test_binding_refusals():
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    ints = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.tree_mask(ints, torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.prefill_tree(torch.zeros(1, 2, 64, dtype=torch.float16), k, k, ints[None], ints, torch.zeros(2, dtype=torch.int32), 1,
                             ints[None])
    with pytest.raises(ValueError, match="CUDA"):
        binding.cache_weigh(torch.zeros(1, 2, 64, dtype=torch.float16), torch.zeros(1, 2), k, k, ints[None], ints)
    with pytest.raises(ValueError, match="CUDA"):
        binding.cache_select(torch.zeros(1, 2, 8), ints, 4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.cache_keep(k, k, ints[None], ints, ints[None, None], ints)
