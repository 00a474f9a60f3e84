"""Which calls the CPython module takes on: ordinary ones must not go through the checks in Python, which cost a call of
a few microseconds half its time again."""
import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

pytestmark = pytest.mark.gpu
H, D, PAGE = 2, 64, 16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


@pytest.fixture
def c_path_only(monkeypatch):
    def no(*args):
        raise AssertionError("the call went through the checks in Python")

    monkeypatch.setattr(binding, "_run", no)


def operands(T=3):
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(T, n, D, generator=g, device="cuda").half() for n in (4, H, H))
    pages = [torch.zeros(8, H, PAGE, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    table = torch.arange(T, dtype=torch.int32, device="cuda")[:, None]
    return q, k, v, *pages, table, torch.full((T,), 5, dtype=torch.int32, device="cuda")


def test_a_table_of_no_angles(c_path_only):
    q, k, v, kp, vp, table, lens = operands()
    out = binding.cache_append(q, k, v, kp, vp, table, lens, rope=torch.empty(40, 0, device="cuda"))
    assert torch.equal(out, q) and torch.equal(kp[:3, :, 4], k) and torch.equal(vp[:3, :, 4], v)


def test_ordinary_calls(c_path_only):
    q, k, v, kp, vp, table, lens = operands()
    rope = binding.rope_table(16, D)
    turned = binding.cache_append(q, k, v, kp, vp, table, lens, rope=rope)
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    out = binding.decode_paged(turned, kp, vp, table, lens)
    assert torch.equal(out, binding.prefill_paged(turned, kp, vp, table, lens, cu, 1))
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.decode_shared(turned, kp, vp, empty, empty, table, lens)


def test_keys_alone(c_path_only):
    _, k, v, kp, vp, table, lens = operands()
    assert binding.cache_append(None, k, v, kp, vp, table, lens) is None
    assert torch.equal(kp[:3, :, 4], k) and torch.equal(vp[:3, :, 4], v)


def test_refusals_of_keys_alone_are_those_of_python():
    q, k, v, kp, vp, table, lens = operands()
    with pytest.raises(ValueError, match="out without q"):
        binding.cache_append(None, k, v, kp, vp, table, lens, out=q)
    with pytest.raises(ValueError):
        binding.cache_append(None, k[:2], v, kp, vp, table, lens)
    with pytest.raises(ValueError):
        binding.cache_append(None, k.float(), v, kp, vp, table, lens)
    with pytest.raises(binding.FaError) as e:
        binding.cache_append(None, k, v, kp, kp, table, lens)
    assert e.value.status == binding.FA_ERR_ALIAS
