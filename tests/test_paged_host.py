"""The paged-cache calls without a GPU: bad arguments come back as the documented status before any CUDA call."""
import pytest

from attention_forward_prefill_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()


def cache(**change):
    a = dict(k_pages=1 << 32, v_pages=2 << 32, page_stride=8 * 64 * 128, head_stride=64 * 128, slot_stride=128, num_pages=100,
             num_heads=8, page_size=64, head_dim=128, dtype=binding.FA_BF16)
    a.update({k: v for k, v in change.items() if k in a})
    return binding.PagedCacheArg(*a.values())


CACHE_REFUSALS = [
    (dict(k_pages=None), binding.FA_ERR_NULL), (dict(v_pages=None), binding.FA_ERR_NULL),
    (dict(num_pages=0), binding.FA_ERR_SHAPE), (dict(num_heads=0), binding.FA_ERR_SHAPE),
    (dict(page_size=8, slot_stride=128), binding.FA_ERR_SHAPE), (dict(page_size=48), binding.FA_ERR_SHAPE),
    (dict(page_size=1 << 21), binding.FA_ERR_SHAPE), (dict(head_dim=96), binding.FA_ERR_HEAD_DIM),
    (dict(dtype=binding.FA_F32), binding.FA_ERR_DTYPE), (dict(k_pages=(1 << 32) + 8), binding.FA_ERR_ALIGN),
    (dict(slot_stride=64), binding.FA_ERR_SHAPE), (dict(slot_stride=0), binding.FA_ERR_SHAPE),
    (dict(slot_stride=-128), binding.FA_ERR_SHAPE), (dict(head_stride=63 * 128), binding.FA_ERR_SHAPE),
    (dict(page_stride=7 * 64 * 128), binding.FA_ERR_SHAPE), (dict(page_stride=8 * 64 * 128 + 4), binding.FA_ERR_ALIGN),
    (dict(page_stride=1 << 40), binding.FA_ERR_SHAPE),
]


def append(**c):
    a = dict(q=3 << 32, k=4 << 32, v=5 << 32, q_out=6 << 32, q_stride=32 * 128, k_stride=8 * 128, v_stride=8 * 128,
             q_out_stride=32 * 128, page_table=7 << 32, max_pages=10, seq_lens=8 << 32, cu=9 << 32, positions=None, B=4, Hq=32,
             total=9, rope=10 << 32, max_positions=640, rope_dim=128, interleaved=0)
    a.update({k: v for k, v in c.items() if k in a})
    return binding.fa_cache_append(cache(**c), *a.values())


@pytest.mark.parametrize("change,status", CACHE_REFUSALS + [
    (dict(k=None), binding.FA_ERR_NULL), (dict(v=None), binding.FA_ERR_NULL), (dict(page_table=None), binding.FA_ERR_NULL),
    (dict(seq_lens=None), binding.FA_ERR_NULL), (dict(q=None), binding.FA_ERR_NULL), (dict(q_out=None), binding.FA_ERR_NULL),
    (dict(Hq=0), binding.FA_ERR_NULL), (dict(rope=None), binding.FA_ERR_NULL),
    (dict(B=0), binding.FA_ERR_SHAPE), (dict(Hq=-1), binding.FA_ERR_SHAPE), (dict(total=-1), binding.FA_ERR_SHAPE),
    (dict(max_pages=0), binding.FA_ERR_SHAPE), (dict(cu=None), binding.FA_ERR_SHAPE), (dict(max_pages=1 << 25), binding.FA_ERR_SHAPE),
    (dict(total=1 << 27), binding.FA_ERR_SHAPE),
    (dict(rope_dim=8), binding.FA_ERR_SHAPE), (dict(rope_dim=144), binding.FA_ERR_SHAPE), (dict(rope_dim=-16), binding.FA_ERR_SHAPE),
    (dict(max_positions=0), binding.FA_ERR_SHAPE), (dict(q_stride=31 * 128), binding.FA_ERR_SHAPE),
    (dict(k_stride=7 * 128), binding.FA_ERR_SHAPE), (dict(v_stride=-1024), binding.FA_ERR_SHAPE),
    (dict(q_out_stride=0), binding.FA_ERR_SHAPE), (dict(k_stride=8 * 128 + 4), binding.FA_ERR_ALIGN),
    (dict(q=(3 << 32) + 2), binding.FA_ERR_ALIGN), (dict(k=(4 << 32) + 8), binding.FA_ERR_ALIGN),
    (dict(rope=(10 << 32) + 4), binding.FA_ERR_ALIGN), (dict(seq_lens=(8 << 32) + 2), binding.FA_ERR_ALIGN),
    (dict(positions=(11 << 32) + 1), binding.FA_ERR_ALIGN), (dict(page_table=(7 << 32) + 1), binding.FA_ERR_ALIGN),
    # what is written overlaps what is read
    (dict(k=(1 << 32) + 1024), binding.FA_ERR_ALIAS), (dict(v=2 << 32), binding.FA_ERR_ALIAS), (dict(q=1 << 32), binding.FA_ERR_ALIAS),
    (dict(q_out=2 << 32), binding.FA_ERR_ALIAS), (dict(q_out=(3 << 32) + 256), binding.FA_ERR_ALIAS),
    (dict(q_out=3 << 32, q_out_stride=33 * 128), binding.FA_ERR_ALIAS), (dict(q_out=4 << 32), binding.FA_ERR_ALIAS),
    (dict(q_out=(8 << 32) - 16), binding.FA_ERR_ALIAS), (dict(page_table=1 << 32), binding.FA_ERR_ALIAS),
    (dict(rope=1 << 32), binding.FA_ERR_ALIAS)])
def test_append_refusals(change, status):
    assert append(**change) == status


def attention(call, **c):
    a = dict(q=3 << 32, out=6 << 32, lse=12 << 32, page_table=7 << 32, max_pages=10, seq_lens=8 << 32, cu=9 << 32, B=4, Hq=32, total=9,
             max_q=5, causal=1, scale=0.1, out_dtype=binding.FA_BF16, ws=None, ws_bytes=0, prefix_table=13 << 32, max_prefix=4,
             prefix_len=14 << 32)
    a.update({k: v for k, v in c.items() if k in a})
    tail = [a[k] for k in ("scale", "out_dtype", "ws", "ws_bytes")]
    if call == "prefill":
        return binding.fa_prefill_paged(cache(**c), *[a[k] for k in (
            "q", "out", "lse", "page_table", "max_pages", "seq_lens", "cu", "B", "Hq", "total", "max_q", "causal")], *tail)
    if call == "decode":
        return binding.fa_decode_paged(cache(**c), *[a[k] for k in (
            "q", "out", "page_table", "max_pages", "seq_lens", "B", "Hq")], *tail)
    return binding.fa_decode_shared(cache(**c), *[a[k] for k in (
        "q", "out", "prefix_table", "max_prefix", "prefix_len", "page_table", "max_pages", "seq_lens", "B", "Hq")], *tail)


COMMON = CACHE_REFUSALS + [
    (dict(q=None), binding.FA_ERR_NULL), (dict(out=None), binding.FA_ERR_NULL), (dict(page_table=None), binding.FA_ERR_NULL),
    (dict(seq_lens=None), binding.FA_ERR_NULL), (dict(B=0), binding.FA_ERR_SHAPE), (dict(Hq=0), binding.FA_ERR_SHAPE),
    (dict(Hq=33), binding.FA_ERR_SHAPE), (dict(max_pages=0), binding.FA_ERR_SHAPE), (dict(max_pages=1 << 24), binding.FA_ERR_SHAPE),
    (dict(B=1 << 26, total=1 << 26), binding.FA_ERR_SHAPE), (dict(out_dtype=7), binding.FA_ERR_DTYPE),
    (dict(q=(3 << 32) + 8), binding.FA_ERR_ALIGN), (dict(out=(6 << 32) + 4), binding.FA_ERR_ALIGN),
    (dict(page_table=(7 << 32) + 2), binding.FA_ERR_ALIGN), (dict(seq_lens=(8 << 32) + 1), binding.FA_ERR_ALIGN),
    (dict(ws=(15 << 32) + 4), binding.FA_ERR_ALIGN), (dict(scale=float("inf")), binding.FA_ERR_SCALE),
    (dict(scale=float("nan")), binding.FA_ERR_SCALE), (dict(out=3 << 32), binding.FA_ERR_ALIAS), (dict(out=1 << 32), binding.FA_ERR_ALIAS),
    (dict(out=2 << 32), binding.FA_ERR_ALIAS), (dict(out=(7 << 32) - 16), binding.FA_ERR_ALIAS), (dict(out=8 << 32), binding.FA_ERR_ALIAS)]


@pytest.mark.parametrize("call", ["decode", "prefill", "shared"])
@pytest.mark.parametrize("change,status", COMMON)
def test_attention_refusals(call, change, status):
    assert attention(call, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(cu=None), binding.FA_ERR_NULL), (dict(total=-1), binding.FA_ERR_SHAPE), (dict(max_q=0), binding.FA_ERR_SHAPE),
    (dict(total=1 << 27), binding.FA_ERR_SHAPE), (dict(max_q=1 << 27), binding.FA_ERR_SHAPE),
    (dict(cu=(9 << 32) + 2), binding.FA_ERR_ALIGN), (dict(lse=(12 << 32) + 2), binding.FA_ERR_ALIGN),
    (dict(lse=6 << 32), binding.FA_ERR_ALIAS), (dict(lse=3 << 32), binding.FA_ERR_ALIAS), (dict(out=9 << 32), binding.FA_ERR_ALIAS)])
def test_prefill_refusals(change, status):
    assert attention("prefill", **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(prefix_table=None), binding.FA_ERR_NULL), (dict(prefix_len=None), binding.FA_ERR_NULL),
    (dict(max_prefix=0), binding.FA_ERR_SHAPE), (dict(max_prefix=1 << 24), binding.FA_ERR_SHAPE),
    (dict(prefix_table=(13 << 32) + 2), binding.FA_ERR_ALIGN), (dict(out=13 << 32), binding.FA_ERR_ALIAS),
    (dict(out=(14 << 32) - 32), binding.FA_ERR_ALIAS)])
def test_shared_refusals(change, status):
    assert attention("shared", **change) == status


def test_strides_that_are_fine_reach_the_device_check():
    """Heads last, K and V in one tensor, and any stride of an extent of one: no argument error is left (the
    call then fails for want of a device, or runs)."""
    fine = (dict(slot_stride=1024, head_stride=128), dict(page_stride=2 * 8 * 64 * 128), dict(num_heads=1, head_stride=3),
            dict(num_pages=1, page_stride=0), dict(q_out=3 << 32), dict(q=None, q_out=None, Hq=0), dict(rope=None, rope_dim=0))
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: only where no device can be reached")
    for change in fine:
        assert append(**change) == binding.FA_ERR_CUDA, change


def test_workspace_sizes_refuse_bad_heads():
    assert binding.fa_paged_workspace_bytes(3, 2, 1, 128) == 0
    assert binding.fa_paged_workspace_bytes(4, 2, 0, 128) == 0
    assert binding.fa_paged_workspace_bytes(4, 2, 1, 80) == 0
    assert binding.fa_shared_workspace_bytes(0, 4, 2, 128) == 0


def test_binding_refusals():
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.decode_paged(torch.zeros(1, 2, 64, dtype=torch.float16), k, k, torch.zeros(1, 1, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        binding.cache_append(None, k[0], k[0], k, k, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
