"""Paged attention at the sizes where the form of a call changes, with ragged lengths, against its definition in 64
bits."""
import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

from .paged_util import Cache, assert_rows, attend

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def queries(T, Hq, d, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(2000 + seed)
    return torch.randn(T, Hq, d, generator=g, device="cuda").to(dtype)


def check(c, q, out, what):
    for b in range(len(c.lens)):
        want, _, bound = attend(q[b:b + 1].double(), *c.keys(b), c.d ** -0.5, False, c.dtype)
        assert_rows(out[b:b + 1], want, bound, f"{what}, sequence {b} of length {c.lens[b]}")


def takes_scratch(call):
    """Whether a call takes memory from the library's pool, as the split form alone does."""
    torch.cuda.synchronize()
    rc, before = binding.fa_pool_stats(reset_high=True)
    call()
    torch.cuda.synchronize()
    rc2, after = binding.fa_pool_stats()
    assert rc == rc2 == binding.FA_OK
    return after[3] > before[2]


# units (B x kv heads) times a cluster's size near the CTAs that run at once
@pytest.mark.parametrize("B", [9, 18, 19, 20, 37, 38, 39])
def test_one_long_sequence_among_short_ones(B):
    """The longest sequence is shared among the SMs at every batch size, and never one cluster's work alone."""
    lens = [8192] + [1 + (i * 29) % 64 for i in range(B - 1)]
    c = Cache(lens, 8, 128, 64, BF16, seed=B, extra_cols=0)
    q = queries(B, 32, 128, BF16)
    out = torch.empty_like(q)

    def call():
        binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, out=out)

    assert takes_scratch(call)
    check(c, q, out, f"batch of {B}")


@pytest.mark.parametrize("units", [35, 36, 37, 38, 71, 72, 74, 76, 142, 143, 152, 153, 285, 286, 304, 305])
@pytest.mark.parametrize("G,d,dtype", [(1, 64, F16), (20, 128, BF16), (64, 64, F16)])
def test_units_that_nearly_fill_the_gpu(units, G, d, dtype):
    lens = [(i * 53) % 260 for i in range(units)]
    c = Cache(lens, 1, d, 32, dtype, seed=units, extra_cols=0)
    q = queries(units, G, d, dtype)
    out = binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens)
    check(c, q, out, f"{units} units")
    assert torch.equal(out, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens))


# 65 to 128 query heads per kv head: the pass over the sequences' own keys runs on tensor-memory tiles too
@pytest.mark.parametrize("cols", [2, 2048])
@pytest.mark.parametrize("prefix", [0, 333, 5000])
@pytest.mark.parametrize("B,G,Hkv,d,dtype", [(5, 65, 1, 64, BF16), (9, 71, 2, 128, F16), (40, 128, 1, 64, F16),
                                             (3, 128, 2, 128, BF16), (1, 100, 1, 128, F16)])
def test_shared_prefix_of_many_heads(B, G, Hkv, d, dtype, prefix, cols):
    lens = [(i * 37) % 200 if i % 3 else 0 for i in range(B)]
    if B > 2:
        lens[-1] = 3000
    c = Cache(lens, Hkv, d, 64, dtype, slots_first=prefix == 333, seed=G, prefix=prefix, extra_cols=cols)
    q = queries(B, G * Hkv, d, dtype)
    out = binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens)
    check(c, q, out, f"prefix {prefix}")
    for _ in range(20):
        assert torch.equal(out, binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens))
