"""Scales at the ends of fp32 in the paged calls (no GPU)."""
import pytest

from attention_forward_prefill_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()


@pytest.mark.parametrize("scale", [2.5e38, -3e38, float("inf"), float("nan")])
def test_scales_whose_log2_units_overflow_are_refused(scale):
    """Scores times an infinite factor would be NaN or 0 x inf."""
    c = binding.PagedCacheArg(1 << 32, 2 << 32, 8 * 64 * 128, 64 * 128, 128, 100, 8, 64, 128, binding.FA_BF16)
    p = [i << 32 for i in range(3, 12)]
    assert binding.fa_decode_paged(c, p[0], p[1], p[2], 10, p[3], 4, 32, scale, binding.FA_BF16) == binding.FA_ERR_SCALE
    assert binding.fa_prefill_paged(c, p[0], p[1], None, p[2], 10, p[3], p[4], 4, 32, 9, 5, 1, scale,
                                    binding.FA_BF16) == binding.FA_ERR_SCALE
    assert binding.fa_decode_shared(c, p[0], p[1], p[5], 4, p[6], p[2], 10, p[3], 4, 32, scale,
                                    binding.FA_BF16) == binding.FA_ERR_SCALE
