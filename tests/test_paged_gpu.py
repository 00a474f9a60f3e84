"""Attention over a paged cache on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

from .paged_util import Cache, assert_rows, attend

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def queries(T, Hq, d, dtype, seed=1, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (torch.randn(T, Hq, d, generator=g, device="cuda") * gain).to(dtype)


def check_decode(c, q, out, scale, what):
    for b in range(len(c.lens)):
        k, v = c.keys(b)
        want, _, bound = attend(q[b:b + 1].double(), k, v, scale, False, c.dtype)
        assert_rows(out[b:b + 1], want, bound, f"{what}, sequence {b} of length {c.lens[b]}")


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 128, 129, 500, 1031]


# A table as wide as the lengths need makes few, short units (clusters); a wide one, with room for
# sequences that are not there, takes the split form with its join.
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,page,dtype,slots_first", [
    (12, 12, 64, 16, F16, False), (14, 2, 64, 16, F16, True), (14, 2, 64, 128, BF16, False),
    (32, 8, 128, 64, BF16, False), (8, 8, 128, 32, F16, True), (64, 8, 128, 256, F16, False),
    (20, 1, 128, 16, BF16, True), (40, 1, 64, 32, BF16, False), (71, 1, 128, 64, F16, True),
    (130, 1, 64, 16, BF16, False), (6, 2, 128, 1024, BF16, False)])
def test_decode_heads_pages_and_lengths(Hq, Hkv, d, page, dtype, slots_first, wide):
    c = Cache(LENS, Hkv, d, page, dtype, slots_first, seed=Hq, extra_cols=(1 << 17) // page if wide else 2)
    q = queries(len(LENS), Hq, d, dtype)
    out = binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens)
    check_decode(c, q, out, d ** -0.5, "decode")
    assert torch.equal(out, binding.decode_paged(q.unsqueeze(2), c.k, c.v, c.table, c.seq_lens).squeeze(2))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens", [[1], [64], [4097], [40000, 3], [0, 0, 0], [0, 9000, 0, 1], [1] * 700, [3, 70] * 2049,
                                  list(range(0, 400, 3))])
def test_decode_batches(lens, wide):
    c = Cache(lens, 2, 128, 64, BF16, seed=len(lens), extra_cols=500 if wide else 1)
    q = queries(len(lens), 8, 128, BF16)
    check_decode(c, q, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens), 128 ** -0.5, "decode")


@pytest.mark.parametrize("dtype,out_dtype", [(F16, F32), (BF16, F32), (F16, BF16), (BF16, F16)])
@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0])
def test_decode_scales_and_output_types(dtype, out_dtype, scale):
    c = Cache([5, 300, 0, 77], 2, 64, 16, dtype, seed=3)
    q = queries(4, 6, 64, dtype)
    out = binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, scale=scale, out_dtype=out_dtype)
    assert out.dtype == out_dtype
    check_decode(c, q, out, scale, f"scale {scale}")


def test_decode_peaked_rows_and_growing_maxima():
    """Scores that rise along the keys move the running maximum at every tile; one key then holds the row."""
    c = Cache([900, 901], 1, 64, 16, F16, seed=5)
    q = queries(2, 4, 64, F16, gain=8.0)
    k = c.rows[0][0]
    k *= torch.linspace(0.1, 4.0, 900, device="cuda", dtype=torch.float64)[:, None, None]
    k.copy_(k.half().double())
    page = c.table[0, :57].long().repeat_interleave(16)[:900]
    c.k[page, :, torch.arange(900, device="cuda") % 16] = k.half()
    check_decode(c, q, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, scale=1.0), 1.0, "peaked")


def test_decode_is_the_same_bits_every_time_and_follows_the_contiguous_cache():
    lens = [777, 12, 2000, 64]
    c = Cache(lens, 4, 128, 32, F16, seed=7)
    q = queries(4, 16, 128, F16)
    first = binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens)
    for _ in range(3):
        assert torch.equal(first, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens))
    flat = torch.zeros(2, 4, 4, 2000, 128, dtype=F16, device="cuda")
    for b, n in enumerate(lens):
        flat[:, b, :, :n] = torch.stack([x.half().transpose(0, 1) for x in c.rows[b]])
    other = binding.decode(q.unsqueeze(2), flat[0], flat[1], c.seq_lens).squeeze(2)
    # both within fp16 weights and one output rounding of the exact rows
    assert (first.float() - other.float()).abs().max() <= 3 * 2.0 ** -11 * float(flat[1].abs().max())


@pytest.mark.parametrize("G,d,dtype", [(32, 128, BF16), (17, 128, F16), (16, 128, BF16), (64, 128, F16), (32, 64, F16)])
def test_many_short_units_keep_their_own_queries(G, d, dtype):
    """Unit after unit through the same shared memory: each one's rows are its own, call after call."""
    lens = [(i * 61) % 450 for i in range(40)]
    c = Cache(lens, 8, d, 64, dtype, seed=21)
    q = queries(40, G * 8, d, dtype)
    out = binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens)
    check_decode(c, q, out, d ** -0.5, "short units")
    for _ in range(200):
        assert torch.equal(out, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens))


def test_offsets_past_32_bits():
    """Pages whose element and byte offsets pass 2^31 and 2^32."""
    Hkv, d, page = 8, 128, 64
    count = (1 << 31) // (Hkv * d * page) + 40  # 2^31 elements and a little
    c = Cache([1000, 70], Hkv, d, page, BF16, seed=9, total_pages=count, behind=0.0)
    assert int(c.table[0, 0]) * Hkv * d * page > 1 << 31
    q = queries(2, 32, d, BF16)
    check_decode(c, q, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens), d ** -0.5, "far pages")
    qp = queries(9, 32, d, BF16, seed=4)
    cu = torch.tensor([0, 8, 9], dtype=torch.int32, device="cuda")
    out = binding.prefill_paged(qp, c.k, c.v, c.table, c.seq_lens, cu, 8, causal=True)
    for b, (lo, hi) in enumerate([(0, 8), (8, 9)]):
        want, _, bound = attend(qp[lo:hi].double(), *c.keys(b), d ** -0.5, True, BF16)
        assert_rows(out[lo:hi], want, bound, f"far pages, chunk {b}")


# ---------------------------------------------------------------- chunks of queries
def check_prefill(lens, new, Hq, Hkv, d, page, dtype, causal, slots_first=False, slack=0, out_dtype=None, scale=None,
                  behind_rows=0, seed=0):
    c = Cache(lens, Hkv, d, page, dtype, slots_first, seed=seed)
    T = sum(new)
    q = queries(T + behind_rows, Hq, d, dtype, seed=seed)
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    lse = torch.full((T + behind_rows, Hq), 7.0, device="cuda")
    out = torch.full((T + behind_rows, Hq, d), 3.0, dtype=out_dtype or dtype, device="cuda")
    got = binding.prefill_paged(q, c.k, c.v, c.table, c.seq_lens, cu, max(new) + slack, causal=causal, scale=scale,
                                out=out, out_dtype=out_dtype, lse=lse)
    assert got is out
    scale = d ** -0.5 if scale is None else scale
    at = 0
    for b, n in enumerate(new):
        want, want_lse, bound = attend(q[at:at + n].double(), *c.keys(b), scale, causal, dtype)
        what = f"sequence {b}: {n} queries on {lens[b]} keys"
        assert_rows(out[at:at + n], want, bound, what)
        none = want_lse == -math.inf
        assert torch.equal(lse[at:at + n] == -math.inf, none), what
        err = (lse[at:at + n].double() - want_lse)[~none].abs()
        # the sum's weights are rounded (u), scores in fp32
        assert err.numel() == 0 or err.max() <= 1.1 * 2.0 ** (-11 if dtype == F16 else -8) + 1e-4, what
        at += n
    assert (out[T:] == 3.0).all() and (lse[T:] == 7.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d,page,dtype,slots_first", [
    (12, 12, 64, 16, F16, False), (14, 2, 64, 32, BF16, True), (32, 8, 128, 64, BF16, False),
    (8, 2, 128, 128, F16, True), (10, 1, 128, 512, BF16, False)])
def test_prefill_ragged(Hq, Hkv, d, page, dtype, slots_first, causal):
    check_prefill([40, 0, 300, 17, 1000, 64, 5], [3, 0, 129, 17, 1, 64, 9], Hq, Hkv, d, page, dtype, causal, slots_first,
                  behind_rows=3)  # the last: more queries than keys, so that the first rows see none when causal


@pytest.mark.parametrize("new,had", [(1, 0), (1, 1), (2, 62), (5, 2000), (64, 64), (127, 1), (128, 128), (255, 0),
                                     (256, 1), (257, 513), (700, 9)])
@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(4, 4, 128, BF16), (14, 2, 64, F16), (8, 1, 128, F16)])
def test_prefill_lengths(new, had, Hq, Hkv, d, dtype):
    check_prefill([new + had], [new], Hq, Hkv, d, 16, dtype, True, slack=5, seed=new)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new", [[3, 9], [300, 1], [1, 700]])
def test_prefill_without_keys(new, causal):
    """Queries of a sequence whose cache is empty give zero rows."""
    check_prefill([0, 0], new, 4, 2, 64, 16, F16, causal)
    check_prefill([0, 40], new, 8, 1, 128, 32, BF16, causal)
    check_prefill([200, 0], new, 3, 3, 128, 64, F16, causal)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_many_and_long(causal):
    check_prefill([20000], [33], 8, 2, 128, 64, BF16, causal)
    check_prefill([1500] * 9, [1500, 1, 0, 700, 1500, 2, 3, 4, 5], 6, 2, 64, 32, F16, causal)
    check_prefill([30] * 300, [i % 7 for i in range(300)], 4, 2, 64, 16, BF16, causal)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.7])
@pytest.mark.parametrize("dtype,out_dtype", [(F16, F32), (BF16, F32), (BF16, F16)])
def test_prefill_scales_and_output_types(scale, dtype, out_dtype):
    check_prefill([333, 90], [100, 90], 6, 2, 128, 32, dtype, True, out_dtype=out_dtype, scale=scale)


def test_prefill_of_one_token_each_is_decode():
    lens = [100, 2, 64, 901]
    c = Cache(lens, 2, 128, 16, BF16, seed=2)
    q = queries(4, 8, 128, BF16)
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    a = binding.prefill_paged(q, c.k, c.v, c.table, c.seq_lens, cu, 1, causal=True)
    assert torch.equal(a, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens))


# ---------------------------------------------------------------- shared prefixes
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("prefix", [0, 1, 64, 333, 5000])
@pytest.mark.parametrize("B,Hq,Hkv,d,page,dtype", [
    (1, 12, 12, 64, 16, F16), (5, 14, 2, 64, 32, BF16), (40, 8, 2, 128, 64, BF16), (300, 4, 1, 64, 16, F16),
    (33, 32, 4, 128, 128, F16), (3, 40, 1, 64, 16, BF16), (2, 140, 1, 64, 16, F16)])
def test_shared_prefix(prefix, B, Hq, Hkv, d, page, dtype, wide):
    lens = [(i * 37) % 200 if i % 5 else 0 for i in range(B)]
    c = Cache(lens, Hkv, d, page, dtype, slots_first=prefix % 2 == 1, seed=B, prefix=prefix,
              extra_cols=(1 << 17) // page if wide else 2)
    q = queries(B, Hq, d, dtype)
    out = binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens)
    # the two passes' rows are joined in fp32: the same bound as one pass
    check_decode(c, q, out, d ** -0.5, f"prefix {prefix}")
    assert torch.equal(out, binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens))


def test_shared_prefix_under_negative_scale_and_other_output():
    c = Cache([9, 0, 70], 2, 64, 16, F16, seed=1, prefix=130)
    q = queries(3, 8, 64, F16)
    out = binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens, scale=-0.3, out_dtype=F32)
    check_decode(c, q, out, -0.3, "negative scale")


# ---------------------------------------------------------------- how it is called
def test_workspaces_streams_and_strides():
    lens = [4000, 50, 1111]
    c = Cache(lens, 2, 128, 64, F16, seed=6, prefix=600)
    q = queries(3, 16, 128, F16)
    want = binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens)
    want_s = binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens)
    need = binding.fa_paged_workspace_bytes(16, 2, 1, 128)
    need_s = binding.fa_shared_workspace_bytes(3, 16, 2, 128)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    ws_s = torch.full((need_s,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(want, binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, workspace=ws))
    assert torch.equal(want_s, binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens,
                                                     workspace=ws_s))
    for small, call in ((ws[:need - 16], lambda w: binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, workspace=w)),
                        (ws_s[:need_s - 16], lambda w: binding.decode_shared(
                            q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens, workspace=w))):
        with pytest.raises(binding.FaError) as e:
            call(small)
        assert e.value.status == binding.FA_ERR_WORKSPACE
    # two streams at once, each from the library's pool
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens))
            outs.append(binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[::2]) and all(torch.equal(o, want_s) for o in outs[1::2])
    # K and V of a page side by side in one tensor, heads last
    both = torch.empty(c.k.shape[0], 64, 2, 2, 128, dtype=F16, device="cuda")
    both[:, :, 0], both[:, :, 1] = c.k.transpose(1, 2), c.v.transpose(1, 2)
    k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    assert torch.equal(want, binding.decode_paged(q, k, v, c.table, c.seq_lens))


@pytest.mark.parametrize("wide", [False, True])
def test_captured_calls_follow_lengths_that_change(wide):
    lens = [300, 5, 0, 129]
    full = Cache([400, 400, 400, 400], 2, 64, 16, BF16, seed=8, prefix=200, extra_cols=8192 if wide else 2)
    q = queries(4, 8, 64, BF16)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]

    def step():
        binding.decode_paged(q, full.k, full.v, full.table, seq, out=outs[0])
        binding.decode_shared(q, full.k, full.v, full.prefix_table, full.prefix_len, full.table, seq, out=outs[1])

    step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for now in (lens, [1, 400, 77, 0], [0, 0, 0, 0], [400, 399, 398, 64]):
        seq.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(now):
            k, v = (x[:n] for x in full.rows[b])
            want, _, bound = attend(q[b:b + 1].double(), k, v, 64 ** -0.5, False, BF16)
            assert_rows(outs[0][b:b + 1], want, bound, f"replayed, length {n}")
            k, v = (torch.cat([f, x]) for f, x in zip(full.front, (k, v)))
            want, _, bound = attend(q[b:b + 1].double(), k, v, 64 ** -0.5, False, BF16)
            assert_rows(outs[1][b:b + 1], want, bound, f"replayed, shared, length {n}")


def test_captured_prefill_beside_an_eager_one():
    """Two graphs, each with scratch of its own, replayed at once on two streams with an eager call between."""
    c = Cache([3000, 700], 2, 128, 64, F16, seed=12, prefix=900, extra_cols=64)
    q, qd = queries(500, 16, 128, F16), queries(2, 16, 128, F16, seed=3)
    cu = torch.tensor([0, 400, 500], dtype=torch.int32, device="cuda")
    calls = (lambda: binding.prefill_paged(q, c.k, c.v, c.table, c.seq_lens, cu, 400, causal=True),
             lambda: binding.decode_paged(qd, c.k, c.v, c.table, c.seq_lens),
             lambda: binding.decode_shared(qd, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens))
    want = [f() for f in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([f() for f in calls])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = [f() for f in calls]
        torch.cuda.synchronize()
        for got in (*outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_python_path_makes_the_same_calls(monkeypatch):
    """What _paged_calls does not take on goes through the checks in Python, to the same result."""
    c = Cache([90, 5, 300], 2, 64, 16, F16, seed=13, prefix=40)
    q = queries(3, 8, 64, F16)
    cu = torch.tensor([0, 1, 1, 3], dtype=torch.int32, device="cuda")
    calls = (lambda **o: binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, **o),
             lambda **o: binding.prefill_paged(q, c.k, c.v, c.table, c.seq_lens, cu, 2, causal=True, **o),
             lambda **o: binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens, **o))
    want = [(f(), f(scale=0.5), f(out=torch.empty_like(q))) for f in calls]

    class Nothing:
        decode = prefill = shared = append = staticmethod(lambda *a: NotImplemented)

    monkeypatch.setattr(binding, "_calls", Nothing)
    for f, (plain, scaled, given) in zip(calls, want):
        assert torch.equal(f(), plain) and torch.equal(f(scale=0.5), scaled) and torch.equal(plain, given)
        assert torch.equal(f(out_dtype=F16), plain)
        wide = f(out_dtype=F32)
        assert wide.dtype == F32 and torch.equal(wide.half(), plain)


def test_binding_refusals():
    c = Cache([90, 5], 2, 64, 16, F16, seed=14, prefix=16)
    q = queries(2, 8, 64, F16)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    good = dict(q=q, k=c.k, v=c.v, table=c.table, lens=c.seq_lens, cu=cu, out=torch.empty_like(q))

    def decode(a):
        binding.decode_paged(a["q"], a["k"], a["v"], a["table"], a["lens"], out=a["out"])

    def prefill(a):
        binding.prefill_paged(a["q"], a["k"], a["v"], a["table"], a["lens"], a["cu"], 1, out=a["out"])

    def shared(a):
        binding.decode_shared(a["q"], a["k"], a["v"], c.prefix_table, c.prefix_len, a["table"], a["lens"], out=a["out"])

    for call in (decode, prefill, shared):
        call(good)
        for change in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(q=q[..., :32]), dict(q=q.transpose(0, 1)),
                       dict(k=c.k.bfloat16()), dict(v=c.v[:-1]), dict(k=c.k[0]), dict(k=c.k.cpu(), v=c.v.cpu()),
                       dict(table=c.table.long()), dict(table=c.table[:1]), dict(table=c.table[0]),
                       dict(table=c.table.cpu()), dict(table=c.table.t()), dict(lens=c.seq_lens.long()),
                       dict(lens=c.seq_lens[:1]), dict(lens=c.seq_lens.cpu()), dict(out=torch.empty_like(q).float()),
                       dict(out=torch.empty_like(q)[:1])):
            if call is prefill and "q" in change and change["q"].shape == q[:1].shape and change["q"].dtype == F16 \
                    and change["q"].is_cuda and change["q"].is_contiguous():
                continue  # fewer packed tokens than the offsets say are recorded on the device, not refused
            with pytest.raises((ValueError, TypeError)):
                call({**good, **change})
        with pytest.raises(binding.FaError) as e:  # seven query heads over two
            call({**good, "q": queries(2, 7, 64, F16), "out": None})
        assert e.value.status == binding.FA_ERR_SHAPE
    for bad in (cu.long(), cu[:2], cu.cpu()):
        with pytest.raises(ValueError):
            prefill({**good, "cu": bad})
    with pytest.raises(binding.FaError) as e:
        binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, scale=float("nan"))
    assert e.value.status == binding.FA_ERR_SCALE
    with pytest.raises(binding.FaError) as e:
        binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens, out=q)
    assert e.value.status == binding.FA_ERR_ALIAS


def test_lengths_and_pages_out_of_range_are_recorded():
    c = Cache([64, 40], 2, 64, 16, F16, seed=4, extra_cols=0)
    q = queries(2, 4, 64, F16)
    assert binding.fa_device_status(True) == 0
    long = torch.tensor([65, -3], dtype=torch.int32, device="cuda")  # the table has 64 slots
    out = binding.decode_paged(q, c.k, c.v, c.table, long)
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN
    want, _, bound = attend(q[:1].double(), *c.keys(0), 0.125, False, F16)
    assert_rows(out[:1], want, bound, "clamped to the table")
    assert (out[1] == 0).all()
    # a page that is none of the cache's: 16 tokens of zero keys and values
    for bad in (-1, c.k.shape[0], 1 << 30):
        table = c.table.clone()
        table[0, 1] = bad
        out = binding.decode_paged(q, c.k, c.v, table, c.seq_lens)
        assert binding.fa_device_status(True) == binding.FA_ERR_PAGE
        k, v = (x.clone() for x in c.keys(0))
        k[16:32], v[16:32] = 0, 0
        want, _, bound = attend(q[:1].double(), k, v, 0.125, False, F16)
        assert_rows(out[:1], want, bound, f"page {bad}")
    cu = torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")
    qp = queries(6, 4, 64, F16)
    binding.prefill_paged(qp, c.k, c.v, c.table, c.seq_lens, cu, 3)
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN
