"""Whole numbers that do not fit the library's 32 bits are refused, not cut off (no GPU)."""
import pytest

from attention_forward_prefill_gb300 import binding, build

BIG = [1 << 31, (1 << 32) + 9, -(1 << 31) - 1, -(1 << 32) + 9, 1 << 70]


@pytest.fixture(scope="module", autouse=True)
def lib():
    pytest.importorskip("torch")
    build.build()
    binding.load()


def paged_calls():
    return [n for n in binding._SIGNATURES if n.startswith(("fa_cache_", "fa_tree_", "fa_prefill_tree", "fa_prefill_paged",
                                                            "fa_decode_paged", "fa_decode_shared"))]


@pytest.mark.parametrize("name", paged_calls())
@pytest.mark.parametrize("value", BIG)
def test_no_argument_is_cut_off(name, value):
    import torch
    types = binding._SIGNATURES[name][1][:-1]  # (the stream is the call's own)
    at = [i for i, t in enumerate(types) if t is binding._i]
    assert at
    for i in at:
        args = [0.5 if t is binding._f else 1 if t is binding._i else None for t in types]
        args[i] = value
        with pytest.raises(binding.FaError, match="FA_ERR_SHAPE"):
            binding._run(name, torch.device("cuda", 0), *args)


@pytest.mark.parametrize("value", BIG + [1 << 30])
def test_no_arrays_of_sizes_that_the_library_refuses(value, monkeypatch):
    """cache_select and tree_mask make their arrays before the library is called."""
    import torch

    class OnDevice(torch.Tensor):  # as far as the checks look
        is_cuda = True

    def no(*args, **kw):
        raise AssertionError("an array was made")

    monkeypatch.setattr(binding, "_calls", binding._InPython)
    monkeypatch.setattr(torch, "empty", no)
    monkeypatch.setattr(torch, "empty_like", no)
    weights = torch.zeros(1, 2, 8).as_subclass(OnDevice)
    lens, cu = (torch.zeros(n, dtype=torch.int32) for n in (1, 2))
    with pytest.raises(binding.FaError, match="FA_ERR_SHAPE"):
        binding.cache_select(weights, lens, value)
    if value > 0:
        with pytest.raises(binding.FaError, match="FA_ERR_SHAPE"):
            binding.tree_mask(torch.zeros(1, dtype=torch.int32).as_subclass(OnDevice), cu, value)
