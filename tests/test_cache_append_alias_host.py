"""Appends whose operands share places (no GPU): refused before any CUDA call, unless nothing that is read or written
twice is shared."""
import itertools

import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

BASE = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()


def append(strides, shape, k_pages, v_pages, q=3 << 42, k=4 << 42, v=5 << 42, q_out=6 << 42, Hq=4, total=9, row_strides=None):
    """shape, strides: (pages, heads, slots, d); pointers in bytes, strides in elements."""
    pages, heads, slots, d = shape
    qs, ks, vs, os = row_strides or (Hq * d, heads * d, heads * d, Hq * d)
    c = binding.PagedCacheArg(k_pages, v_pages, *strides, pages, heads, slots, d, binding.FA_F16)
    return binding.fa_cache_append(c, q, k, v, q_out, qs, ks, vs, os, 7 << 42, 10, 8 << 42, 9 << 42, None, 4, Hq, total,
                                   None, 0, 0, 0)


def accepted(rc):
    """No argument error: the call fails for want of a device (where there is one, it is not made)."""
    return rc == binding.FA_ERR_CUDA


skip_on_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@skip_on_gpu
@pytest.mark.parametrize("order", list(itertools.permutations(["page", "head", "slot"])))
@pytest.mark.parametrize("d,gap", [(64, 0), (128, 64)])
def test_a_slots_key_and_value_are_two_places(order, d, gap):
    """Against the places themselves, for V at every 8-element offset around K."""
    n = dict(page=3, head=2, slot=16)
    stride, at = {}, 2 * d if gap else d  # (room for the other tensor's rows between)
    for name in order:
        stride[name] = at
        at = at * n[name] + gap
    where = [(i * stride["page"] + j * stride["head"] + s * stride["slot"]) for i in range(3) for j in range(2) for s in range(16)]
    starts = set(where)
    free = taken = 0
    for delta in list(range(-3 * d, 3 * d + 1, 8)) + [x + e for x in (max(where), -max(where), stride["head"], stride["page"])
                                                      for e in (-d, -8, 0, 8, d)]:
        # two rows of d share a place when they start less than d apart
        shared = any(w + delta + e in starts for w in where for e in range(-d + 8, d, 8))
        rc = append((stride["page"], stride["head"], stride["slot"]), (3, 2, 16, d), BASE, BASE + 2 * delta)
        assert rc == binding.FA_ERR_ALIAS if shared else accepted(rc), (delta, rc)
        taken, free = taken + shared, free + (not shared)
    assert taken and free


@skip_on_gpu
def test_key_and_value_in_one_tensor_are_fine():
    H, S, d = 8, 16, 64
    for strides, off in (((2 * H * S * d, S * d, d), H * S * d),      # [page][2][head][slot][d]
                         ((2 * H * S * d, 2 * S * d, d), S * d),      # [page][head][2][slot][d]
                         ((2 * H * S * d, d, 2 * H * d), H * d)):     # [page][slot][2][head][d]
        assert accepted(append(strides, (5, H, S, d), BASE, BASE + 2 * off))
        assert append(strides, (5, H, S, d), BASE, BASE) == binding.FA_ERR_ALIAS
    assert append((0, S * d, d), (1, H, S, d), BASE, BASE + 2 * d) == binding.FA_ERR_ALIAS


@skip_on_gpu
@pytest.mark.parametrize("total", [1, 2, 9])
def test_in_place_leaves_keys_and_values_alone(total):
    """q turned in place: k and v may lie between its rows and not on them."""
    Hq, H, d = 4, 2, 64
    pages = ((H * 16 * d, 16 * d, d), (5, H, 16, d), BASE, 2 * BASE)
    fused = (Hq + 2 * H) * d
    q = 1 << 44

    def call(k_off, v_off, k_stride=fused, v_stride=fused):
        return append(*pages, q=q, q_out=q, k=q + 2 * k_off, v=q + 2 * v_off, total=total,
                      row_strides=(fused, k_stride, v_stride, fused))

    assert accepted(call(Hq * d, (Hq + H) * d))
    assert accepted(call(Hq * d - fused, (Hq + H) * d - fused))     # the rows of the token before
    assert accepted(call(total * fused, -total * fused))
    far = (total + 3) * fused
    assert accepted(call(far, -far))
    for k, v in ((0, far), (far, 0), (Hq * d - 8, far), (far, 8 - H * d), ((total - 1) * fused, far),
                 (far, (total - 1) * fused + Hq * d - 8), (-(total - 1) * fused, far)):
        assert call(k, v) == binding.FA_ERR_ALIAS, (k, v)
    # rows one over on each side
    if total > 1:
        assert call(fused - 8, far) == binding.FA_ERR_ALIAS
        assert call(Hq * d, far, k_stride=fused + 64) == binding.FA_ERR_ALIAS  # other strides: by their spans
    assert accepted(append(*pages, q=q, q_out=q, k=1 << 45, v=1 << 45, total=total, row_strides=(fused, fused, fused, fused)))
