"""Scales so small that fp32 keeps them as subnormals: every visible key weighs the same, in every form of the call."""
import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

from .paged_util import Cache, assert_rows, attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()


@pytest.mark.parametrize("scale", [1e-39, -1e-39, 2e-45, 1.2e-38, -8e-39])
@pytest.mark.parametrize("new,d,dtype", [(1, 64, torch.float16), (9, 128, torch.bfloat16), (150, 128, torch.bfloat16),
                                         (150, 64, torch.float16)])
def test_subnormal_scales(new, d, dtype, scale):
    lens = [333, 200]
    c = Cache(lens, 2, d, 16, dtype, seed=new)
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(2 * new, 4, d, generator=g, device="cuda").to(dtype)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    lse = torch.empty(2 * new, 4, device="cuda")
    out = binding.prefill_paged(q, c.k, c.v, c.table, c.seq_lens, cu, new, causal=True, scale=scale, lse=lse)
    for b in range(2):
        rows = slice(b * new, (b + 1) * new)
        want, want_lse, bound = attend(q[rows].double(), *c.keys(b), scale, True, dtype)
        assert_rows(out[rows], want, bound, f"scale {scale}, sequence {b}")
        assert (lse[rows].double() - want_lse).abs().max() <= 1e-4  # every weight is 1: no rounding of weights
