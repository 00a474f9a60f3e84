"""The device status word when a call clamped an offset before another's wait ran out."""
import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()


@pytest.mark.parametrize("watchdog_first", [False, True])
def test_a_wait_that_ran_out_wins_over_clamped_offsets(watchdog_first):
    q, k, v = (torch.randn(300, h, 64, device="cuda").half() for h in (4, 2, 2))
    out = torch.zeros_like(q)
    cu = torch.tensor([0, 200, 150], dtype=torch.int32, device="cuda")  # decreasing: clamped and recorded
    result = torch.zeros(4, dtype=torch.int64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def clamped():
        assert binding.fa_prefill_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), cu.data_ptr(), cu.data_ptr(),
                                         2, 4, 2, 300, 300, 200, 200, 64, 1, 0.125, binding.FA_F16, binding.FA_F16, 0,
                                         stream) == binding.FA_OK

    def ran_out():  # a wait on a barrier that nothing arrives at, given up after a millisecond
        assert binding.fa_watchdog_selftest(1_000_000, result.data_ptr(), stream) == binding.FA_OK

    assert binding.fa_device_status(True) == 0
    for call in (ran_out, clamped) if watchdog_first else (clamped, ran_out):
        call()
    assert binding.fa_device_status(True) == binding.FA_ERR_WATCHDOG
    assert binding.fa_device_status(True) == 0
