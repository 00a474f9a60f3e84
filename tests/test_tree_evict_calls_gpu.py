"""The calls for drafted trees and eviction on torch tensors: ordinary ones are read by the CPython module, the checks in
Python make the same calls, and both refuse the same arguments."""
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


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def operands():
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(5, 4, D, generator=g, device="cuda").half()
    pages = [torch.randn(9, H, PAGE, D, generator=g, device="cuda").half() for _ in range(2)]
    return dict(q=q, k=pages[0], v=pages[1], table=torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3),
                lens=ints(40, 7, 20), cu=ints(0, 3, 3, 5), parents=ints(-1, 0, 0, -1, 0), lse=torch.full((5, 4), 3.0, device="cuda"),
                weights=torch.rand(3, H, 48, generator=g, device="cuda"), keep=ints(*range(1, 7)).view(3, 1, 2), counts=ints(2, 1, 2))


def all_calls(o, make):
    """Each call with what `make` gives to its output: results that can be compared."""
    mask, positions = binding.tree_mask(o["parents"], o["cu"], 3, o["lens"])
    out = [mask, positions, binding.tree_mask(o["parents"], o["cu"], 3)[0]]
    lse = torch.empty_like(o["lse"])
    out.append(binding.prefill_tree(o["q"], o["k"], o["v"], o["table"], o["lens"], o["cu"], 3, mask, scale=0.2, lse=lse))
    out += [lse, binding.prefill_tree(o["q"], o["k"], o["v"], o["table"], o["lens"], o["cu"], 3, mask, out=make(o["q"]))]
    lse = torch.empty_like(o["lse"])
    out += [binding.prefill_paged(o["q"], o["k"], o["v"], o["table"], o["lens"], o["cu"], 3, causal=True, lse=lse), lse]
    for w in (o["weights"], None):
        out.append(binding.cache_weigh(o["q"], o["lse"], o["k"], o["v"], o["table"], o["lens"], o["cu"], 3, weights=w, decay=0.5,
                                       out=torch.zeros_like(o["weights"])))
    out.append(binding.cache_weigh(o["q"][:3], o["lse"][:3], o["k"], o["v"], o["table"], o["lens"], weights=o["weights"].clone(),
                                   scale=0.1, causal=False, out=torch.zeros_like(o["weights"])))
    out += binding.cache_select(o["weights"], o["lens"], 9, sink=1, recent=2)
    k, v = o["k"].clone(), o["v"].clone()
    out += binding.cache_keep(k, v, o["table"], o["lens"], o["keep"], o["counts"])
    k, v = o["k"].clone(), o["v"].clone()
    out += binding.cache_keep(k, v, o["table"], o["lens"], o["keep"], o["counts"], first=ints(0, 1, 1), out_table=o["table"])
    return out


def test_ordinary_calls_do_not_go_through_the_checks_in_python(monkeypatch):
    o = operands()

    def no(*args):
        raise AssertionError("the call went through the checks in Python")

    monkeypatch.setattr(binding, "_run", no)
    all_calls(o, torch.empty_like)


def test_the_python_path_makes_the_same_calls(monkeypatch):
    o = operands()
    want = all_calls(o, torch.empty_like)
    monkeypatch.setattr(binding, "_calls", binding._InPython)
    got = all_calls(o, torch.empty_like)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("in_python", [False, True])
def test_refusals(monkeypatch, in_python):
    o = operands()
    if in_python:
        monkeypatch.setattr(binding, "_calls", binding._InPython)
    mask = ints(1, 1, 1, 1, 1)[:, None]
    tree = lambda **c: binding.prefill_tree(*[c.get(k, v) for k, v in dict(  # noqa: E731
        q=o["q"], k=o["k"], v=o["v"], table=o["table"], lens=o["lens"], cu=o["cu"], most=3, mask=mask).items()], lse=c.get("lse"))
    weigh = lambda **c: binding.cache_weigh(*[c.get(k, v) for k, v in dict(  # noqa: E731
        q=o["q"], lse=o["lse"], k=o["k"], v=o["v"], table=o["table"], lens=o["lens"], cu=o["cu"], most=3).items()],
        weights=c.get("weights"), out=c.get("out"), decay=c.get("decay", 1.0))
    keep = lambda **c: binding.cache_keep(*[c.get(k, v) for k, v in dict(  # noqa: E731
        k=o["k"], v=o["v"], table=o["table"], lens=o["lens"], keep=o["keep"], counts=o["counts"]).items()],
        first=c.get("first"), out_table=c.get("out_table"))
    for bad in (dict(q=o["q"].bfloat16()), dict(q=o["q"][:, :, ::2]), dict(q=o["q"].cpu()), dict(cu=o["cu"][:-1].contiguous()), dict(cu=o["cu"].long()),
                dict(mask=mask[:4]), dict(mask=mask[:, 0]), dict(mask=mask.long()), dict(mask=mask.expand(5, 2)), dict(lse=o["lse"].double()),
                dict(lse=o["lse"][:4]), dict(v=o["v"][:8]), dict(table=o["table"][:2].contiguous())):
        with pytest.raises(ValueError):
            tree(**bad)
    for bad in (dict(most=0), dict(most=33)):
        with pytest.raises(binding.FaError, match="SHAPE"):
            tree(**bad)
    w = o["weights"]
    for bad in (dict(q=o["q"].float()), dict(lse=o["lse"][:, :3]), dict(lse=o["lse"].half()), dict(cu=None), dict(cu=o["cu"][1:].contiguous()),
                dict(weights=w.double()), dict(weights=w[:, :1]), dict(weights=w[:, :, ::2]), dict(out=w[:2]), dict(weights=w, out=w[:, :, :40].contiguous()),
                dict(weights=w.cpu()), dict(out=w[0])):
        with pytest.raises(ValueError):
            weigh(**bad)
    with pytest.raises(binding.FaError, match="SCALE"):
        weigh(decay=float("nan"), out=w.clone())
    with pytest.raises(binding.FaError, match="ALIAS"):
        flat = torch.zeros(2 * w.numel(), device="cuda")
        weigh(weights=flat[:w.numel()].view(w.shape), out=flat[4:4 + w.numel()].view(w.shape))
    for bad in (dict(weights=w.half()), dict(weights=w.cpu()), dict(weights=w[0]), dict(weights=w.transpose(1, 2)), dict(lens=o["lens"][:2]),
                dict(lens=o["lens"].long())):
        with pytest.raises(ValueError):
            binding.cache_select(bad.get("weights", w), bad.get("lens", o["lens"]), 9)
    for bad in ((0, 0, 0), (9, 5, 5), (9, -1, 0), (9, 0, -1)):
        with pytest.raises(binding.FaError, match="SHAPE"):
            binding.cache_select(w, o["lens"], bad[0], sink=bad[1], recent=bad[2])
    many = ints(*range(9)).view(3, 3, 1)
    for bad in (dict(keep=many), dict(keep=o["keep"].long()), dict(keep=o["keep"][:2]), dict(keep=o["keep"][:, 0]), dict(counts=o["counts"][:2]),
                dict(first=o["counts"].long()), dict(first=o["counts"][:2]), dict(out_table=o["table"][:2]), dict(out_table=o["counts"]),
                dict(v=o["v"].bfloat16())):
        with pytest.raises(ValueError):
            keep(**bad)
    for bad in (dict(parents=o["parents"].long()), dict(cu=o["cu"].long()), dict(cu=o["cu"].cpu()), dict(lens=o["lens"][:2])):
        with pytest.raises(ValueError):
            binding.tree_mask(bad.get("parents", o["parents"]), bad.get("cu", o["cu"]), 3, bad.get("lens"))
    for most, cu in ((0, o["cu"]), (3, o["cu"][:1])):
        with pytest.raises(binding.FaError, match="SHAPE"):
            binding.tree_mask(o["parents"], cu, most)


def test_calls_without_anything_to_do():
    o = operands()
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    mask, positions = binding.tree_mask(o["parents"][:0], none, 3, o["lens"])
    assert mask.shape == (0, 1) and positions.shape == (0,)
    assert binding.prefill_tree(o["q"][:0], o["k"], o["v"], o["table"], o["lens"], none, 3, mask).shape == (0, 4, D)
    w = o["weights"].clone()
    binding.cache_weigh(o["q"][:0], o["lse"][:0], o["k"], o["v"], o["table"], o["lens"], none, 3, weights=w, decay=0.5, out=w)
    assert torch.equal(w, o["weights"])
    fresh = binding.cache_weigh(o["q"][:0], o["lse"][:0], o["k"], o["v"], o["table"], o["lens"], none, 30)
    assert fresh.shape == (3, H, 48) and not fresh.any()
    k, v = o["k"].clone(), o["v"].clone()
    binding.cache_keep(k, v, o["table"], o["lens"], o["keep"][:, :, :0], o["counts"])
    binding.cache_keep(k, v, o["table"], o["lens"], o["keep"], o["counts"] * 0)
    assert torch.equal(k, o["k"]) and torch.equal(v, o["v"])


def test_other_streams_see_what_theirs_has_made():
    """Inputs that a stream makes right before the calls, which then run on that stream."""
    o = operands()
    want = all_calls(o, torch.empty_like)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        late = {n: t.clone() for n, t in o.items()}
        got = all_calls(late, torch.empty_like)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
