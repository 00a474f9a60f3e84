"""cache_append on the GPU against its definition in 64 bits, and a serving loop over all the paged calls."""
import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

from .paged_util import U, assert_rows, attend

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def turned(x, pos, rot, inter, base=10000.0):
    """x [T, H, d] float64 at positions pos."""
    if not rot:
        return x.clone()
    a = pos.double()[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    c, s = a.cos()[:, None], a.sin()[:, None]
    y = x.clone()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    return y


def assert_turned(got, want, size, what):
    """One rounding to 16 bits, and fp32 products of a table that is rounded to fp32 itself."""
    err = (got.double() - want).abs()
    tol = U[got.dtype] * want.abs() * 1.001 + 2.0 ** -22 * size + (2.0 ** -25 if got.dtype == F16 else 2.0 ** -133)
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())} of {err.numel()} off, worst {float((err - tol).max()):.3e}"


class Step:
    """New tokens of a batch and an empty cache to put them in."""

    def __init__(self, new, lens, Hq, Hkv, d, page, dtype, slots_first=False, fused=False, behind=0, seed=0, extra=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        T = sum(new) + behind
        need = [-(-n // page) for n in lens]
        count = sum(need) + extra
        order = torch.randperm(count, generator=g, device="cuda").tolist()
        cols = max(need + [1]) + 1
        self.table_rows, at = [], 0
        for n in need:
            self.table_rows.append(order[at:at + n] + [-5] * (cols - n))
            at += n
        self.table = ints(self.table_rows)
        self.new, self.lens, self.d, self.page, self.T = new, lens, d, page, T
        self.seq_lens, self.cu = ints(lens), ints([0] + torch.tensor(new).cumsum(0).tolist())
        if fused:
            qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device="cuda").to(dtype)
            self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = (torch.randn(T, h, d, generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
        shape = (count, page, Hkv, d) if slots_first else (count, Hkv, page, d)
        raw = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2)]
        self.kp, self.vp = (x.transpose(1, 2) if slots_first else x for x in raw)

    def want(self, rot, inter, positions=None):
        kp, vp, q = self.kp.double(), self.vp.double(), torch.zeros_like(self.q, dtype=torch.float64)
        pos = torch.cat([torch.arange(n - a, n, device="cuda") for a, n in zip(self.new, self.lens)] +
                        [torch.zeros(0, device="cuda", dtype=torch.int64)])
        T = pos.numel()
        angle = pos if positions is None else positions[:T]
        k, v = turned(self.k[:T].double(), angle, rot, inter), self.v[:T].double()
        q = turned(self.q[:T].double(), angle, rot, inter)
        seq = torch.repeat_interleave(torch.arange(len(self.new), device="cuda"), torch.tensor(self.new, device="cuda"))
        page = self.table[seq, pos // self.page].long()
        kp[page, :, pos % self.page], vp[page, :, pos % self.page] = k, v
        touched = torch.zeros(self.kp.shape[0], self.page, dtype=torch.bool, device="cuda")
        touched[page, pos % self.page] = True
        return q, kp, vp, touched

    def run(self, rope, inter, out=None, positions=None, cu=True):
        return binding.cache_append(self.q, self.k, self.v, self.kp, self.vp, self.table, self.seq_lens,
                                    cu_seqlens=self.cu if cu else None, rope=rope, interleaved=inter, positions=positions,
                                    out=out)

    def check(self, rot, inter, base_rows=None, positions=None, cu=True, what=""):
        want_q, want_k, want_v, touched = self.want(rot, inter, positions)
        before = self.kp.clone(), self.vp.clone()
        rope = binding.rope_table(base_rows or max(self.lens + [1]), rot) if rot else None
        out = torch.full((self.T,) + self.q.shape[1:], 9.0, dtype=self.q.dtype, device="cuda")
        q_in = self.q.double()
        got = self.run(rope, inter, out, positions, cu)
        T = want_q.shape[0]
        big = float(max(self.q.abs().max(), self.k.abs().max())) * 2
        assert_turned(got[:T], want_q, big, what + " q")
        assert (got[T:] == 9.0).all()
        assert_turned(self.kp, want_k, big, what + " k")
        assert torch.equal(self.vp.double(), want_v)
        same = ~touched[:, None, :, None].expand_as(self.kp)
        assert torch.equal(self.kp[same], before[0][same])  # every other slot as it was
        if rot < self.d:
            assert torch.equal(got[:T, :, rot:].double(), q_in[:T, :, rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,page,dtype,rot,slots_first,fused", [
    (12, 12, 64, 16, F16, 64, False, False), (14, 2, 64, 32, BF16, 32, True, True), (32, 8, 128, 64, BF16, 128, False, True),
    (8, 1, 128, 128, F16, 96, True, False), (1, 1, 64, 16, F16, 16, False, False), (7, 7, 128, 256, BF16, 0, False, True)])
def test_tokens_reach_their_slots_turned(Hq, Hkv, d, page, dtype, rot, slots_first, fused, inter):
    new, lens = [1, 0, 33, 5, 200, 1], [17, 9, 33, 1000, 263, 1]
    Step(new, lens, Hq, Hkv, d, page, dtype, slots_first, fused, behind=2, seed=rot).check(rot, inter)


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 257, 1100])
def test_one_token_each(B):
    lens = [1 + (i * 13) % 70 for i in range(B)]
    for cu in (True, False):
        Step([1] * B, lens, 6, 2, 64, 16, BF16, seed=B).check(64, False, cu=cu)


def test_empty_sequences_everywhere():
    new = [0] * 5 + [2] + [0] * 40 + [3] + [0] * 7
    lens = [n + 4 for n in new]
    Step(new, lens, 4, 2, 64, 16, F16).check(64, True)
    Step([0, 0], [3, 0], 4, 2, 64, 16, F16, behind=4).check(64, True)


def test_positions_of_their_own_and_in_place():
    s = Step([3, 1, 4], [3, 40, 20], 4, 2, 128, 16, BF16, fused=True, behind=1)
    pos = ints([100000, 7, 0, 131071, 5, 6, 65536, 1, 0])
    want_q, want_k, want_v, _ = s.want(128, False, pos)
    rope = binding.rope_table(131072, 128)
    keep = s.q[8].clone()
    got = s.run(rope, False, out=s.q, positions=pos)
    assert got.data_ptr() == s.q.data_ptr()
    assert_turned(s.q[:8], want_q, 16.0, "in place")
    assert torch.equal(s.q[8], keep)
    assert_turned(s.kp, want_k, 16.0, "k")
    assert torch.equal(s.vp.double(), want_v)


def test_keys_alone():
    s = Step([2, 3], [2, 10], 4, 2, 64, 16, F16)
    _, want_k, want_v, _ = s.want(64, False)
    assert binding.cache_append(None, s.k, s.v, s.kp, s.vp, s.table, s.seq_lens, cu_seqlens=s.cu,
                                rope=binding.rope_table(64, 64)) is None
    assert_turned(s.kp, want_k, 16.0, "k")
    assert torch.equal(s.vp.double(), want_v)


def test_the_python_path_makes_the_same_calls_and_refuses(monkeypatch):
    def both():
        s = Step([3, 0, 2], [3, 9, 40], 4, 2, 64, 16, F16, fused=True, seed=4)
        return s, s.run(binding.rope_table(64, 48), True)

    one, first = both()

    class Nothing:
        append = staticmethod(lambda *a: NotImplemented)

    real = binding._calls
    monkeypatch.setattr(binding, "_calls", Nothing)
    two, second = both()
    assert torch.equal(first, second) and torch.equal(one.kp, two.kp) and torch.equal(one.vp, two.vp)
    for fast in (real, Nothing):
        monkeypatch.setattr(binding, "_calls", fast)
        s = Step([3, 0, 2], [3, 9, 40], 4, 2, 64, 16, F16, seed=4)
        good = dict(q=s.q, k=s.k, v=s.v, kp=s.kp, vp=s.vp, table=s.table, lens=s.seq_lens, cu=s.cu,
                    rope=binding.rope_table(64, 64), positions=None, out=None)

        def call(a):
            return binding.cache_append(a["q"], a["k"], a["v"], a["kp"], a["vp"], a["table"], a["lens"], cu_seqlens=a["cu"],
                                        rope=a["rope"], positions=a["positions"], out=a["out"])

        call(good)
        for change in (dict(q=s.q.float()), dict(q=s.q[:1]), dict(k=s.k[:1]), dict(v=s.v[:, :1]), dict(k=s.k.cpu()),
                       dict(k=s.k.transpose(0, 1)), dict(q=s.q[..., :32]), dict(kp=s.kp.bfloat16()), dict(vp=s.vp[:1]),
                       dict(table=s.table[:1]), dict(lens=s.seq_lens.long()), dict(cu=s.cu[:2]), dict(cu=s.cu.long()),
                       dict(rope=good["rope"].double()), dict(rope=good["rope"][0]), dict(rope=good["rope"].t()),
                       dict(positions=s.cu), dict(out=s.q[:1]), dict(out=s.q.float()), dict(q=None, out=s.q)):
            with pytest.raises(ValueError):
                call({**good, **change})
        for change, status in ((dict(rope=binding.rope_table(64, 80)), binding.FA_ERR_SHAPE),
                               (dict(rope=binding.rope_table(64, 8)), binding.FA_ERR_SHAPE),
                               (dict(cu=None), binding.FA_ERR_SHAPE), (dict(out=s.q[:, :4].clone()[:, :4]), None)):
            if status is None:
                call({**good, **change})
                continue
            with pytest.raises(binding.FaError) as e:
                call({**good, **change})
            assert e.value.status == status


def test_no_tokens():
    s = Step([0, 0], [3, 0], 4, 2, 64, 16, F16)
    before = s.kp.clone()
    out = s.run(binding.rope_table(8, 64), False)
    assert out.shape == (0, 4, 64) and torch.equal(s.kp, before)


def test_slots_past_32_bits():
    Hkv, d, page = 8, 128, 64
    count = (1 << 31) // (Hkv * d * page) + 8
    kp, vp = (torch.zeros(count, Hkv, page, d, dtype=BF16, device="cuda") for _ in range(2))
    k, v = (torch.randn(3, Hkv, d, device="cuda").to(BF16) for _ in range(2))
    table, lens = ints([[count - 1]]), ints([9])
    assert (count - 1) * Hkv * page * d > 1 << 31
    binding.cache_append(None, k, v, kp, vp, table, lens, cu_seqlens=ints([0, 3]))
    assert torch.equal(kp[-1, :, 6:9], k.transpose(0, 1)) and torch.equal(vp[-1, :, 6:9], v.transpose(0, 1))
    assert int(kp[:-1].count_nonzero()) == 0 and int(kp[-1, :, :6].count_nonzero()) == 0


def test_positions_and_pages_out_of_range_are_recorded():
    assert binding.fa_device_status(True) == 0
    rope = binding.rope_table(32, 64)
    for change, status in ((dict(seq_lens=ints([0, 4])), binding.FA_ERR_SEQ_LEN),        # position -1
                           (dict(seq_lens=ints([33, 4])), binding.FA_ERR_SEQ_LEN),       # behind the table's 32 slots
                           (dict(table=ints([[-1, 0], [1, -1]])), binding.FA_ERR_PAGE),
                           (dict(table=ints([[4, 0], [1, -1]])), binding.FA_ERR_PAGE)):
        s = Step([1, 2], [5, 4], 4, 2, 64, 16, F16, extra=2)
        before = s.kp.clone()
        _, want_k, _, _ = s.want(64, False)
        for name, value in change.items():
            setattr(s, name, value)
        if "table" in change:
            page = 1
        else:
            page = s.table_rows[1][0]
        s.table = s.table if "table" in change else ints([r[:2] for r in s.table_rows])
        s.run(rope, False)
        assert binding.fa_device_status(True) == status
        # the other sequence's tokens are there, the first one's nowhere
        want = before.double()
        want[page, :, 2:4] = turned(s.k[1:3].double(), ints([2, 3]), 64, False).transpose(0, 1)
        assert_turned(s.kp, want, 16.0, "others")
    s = Step([1], [30], 4, 2, 64, 16, F16)
    s.run(binding.rope_table(8, 64), False)  # the position is behind the angle table
    assert binding.fa_device_status(True) == binding.FA_ERR_SEQ_LEN


@pytest.mark.parametrize("shared", [False, True])
def test_serving_loop(shared):
    """A batch's prompts in two chunks, then captured single-token steps: append, attention, lengths moved on."""
    Hq, Hkv, d, page, dtype, B = 8, 2, 64, 16, BF16, 3
    prompt, steps, front = [37, 1, 80], 5, 50 if shared else 0
    g = torch.Generator(device="cuda").manual_seed(1)
    count, cols = 40, 8
    kp, vp = (torch.full((count, Hkv, page, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table, prefix_table = order[:B * cols].view(B, cols).contiguous(), order[B * cols:B * cols + 4].contiguous()
    prefix_len = ints([front])
    rope = binding.rope_table(256, d)
    fresh = lambda T: [torch.randn(T, h, d, generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv)]  # noqa: E731
    K, V = [[] for _ in range(B)], [[] for _ in range(B)]
    pre_k = pre_v = torch.zeros(0, Hkv, d, device="cuda", dtype=torch.float64)
    if shared:
        _, k, v = fresh(front)
        binding.cache_append(None, k, v, kp, vp, prefix_table[None], ints([front]), cu_seqlens=ints([0, front]), rope=rope)
        pre_k = turned(k.double(), torch.arange(front, device="cuda"), d, False).to(dtype).double()
        pre_v = v.double()
    lens = [0] * B

    def check(q, out, b, rows, pos, what):
        if not pos.numel():
            return
        k = torch.cat([pre_k] + K[b])
        v = torch.cat([pre_v] + V[b])
        qt = turned(q[rows].double(), pos, d, False).to(dtype).double()
        want, _, bound = attend(qt, k, v, d ** -0.5, True, dtype)
        # a turned q or k may round the other way than here (an fp32 table): one step, 2 u, of its own size
        assert_rows(out[rows], want, bound + 4 * U[dtype] * v.abs().max(), what)

    for part in (0, 1):
        new = [n - n // 2 if part else n // 2 for n in prompt]
        lens = [a + n for a, n in zip(lens, new)]
        cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist())
        q, k, v = fresh(sum(new))
        pos = torch.cat([torch.arange(n - a, n, device="cuda") for a, n in zip(new, lens)]) + front
        q_out = binding.cache_append(q, k, v, kp, vp, table, ints(lens), cu_seqlens=cu.int().cuda(), rope=rope,
                                     positions=pos.int())
        for b in range(B):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            K[b].append(turned(k[rows].double(), pos[rows], d, False).to(dtype).double())
            V[b].append(v[rows].double())
        if not shared:
            out = binding.prefill_paged(q_out, kp, vp, table, ints(lens), cu.int().cuda(), max(new), causal=True)
            for b in range(B):
                rows = slice(int(cu[b]), int(cu[b + 1]))
                check(q, out, b, rows, pos[rows], f"prompt part {part}, sequence {b}")
    seq = ints(lens)
    q, k, v = fresh(B)
    positions = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)

    def step():
        seq.add_(1)
        torch.add(seq, front - 1, out=positions)
        q_out = binding.cache_append(q, k, v, kp, vp, table, seq, rope=rope, positions=positions)
        if shared:
            binding.decode_shared(q_out, kp, vp, prefix_table, prefix_len, table, seq, out=out)
        else:
            binding.decode_paged(q_out, kp, vp, table, seq, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once outside the capture, then the lengths back
        step()
    torch.cuda.synchronize()
    seq.sub_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for t, x in zip((q, k, v), fresh(B)):
            t.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        assert seq.tolist() == lens
        for b in range(B):
            pos = torch.tensor([front + lens[b] - 1], device="cuda")
            K[b].append(turned(k[b:b + 1].double(), pos, d, False).to(dtype).double())
            V[b].append(v[b:b + 1].double())
            check(q, out, b, slice(b, b + 1), pos, f"step {i}, sequence {b}")


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("wide", [1, 400])
def test_a_chain_of_dependent_calls_needs_no_waiting(shared, wide):
    """Each step's queries, keys and values come from the last step's rows, nothing waits on the host, and kernels
    start under the tail of those before them: the same bits as with a wait after every call."""
    Hq, Hkv, d, page, B, steps, front = 16, 4, 128, 32, 6, 40, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    cols = -(-(steps + 60) // page)
    start = torch.randn(B, Hq, d, generator=g, device="cuda").to(BF16)
    pre = [torch.randn(front, Hkv, d, generator=g, device="cuda").to(BF16) for _ in range(2)]
    rope = binding.rope_table(1024, d)
    table = torch.full((B, cols * wide), -1, dtype=torch.int32, device="cuda")
    table[:, :cols] = torch.randperm(B * cols, generator=g, device="cuda").view(B, cols).int()
    front_table = (B * cols + torch.arange(-(-front // page), device="cuda")).int()

    def run(wait):
        kp, vp = (torch.zeros(B * cols + 10, Hkv, page, d, dtype=BF16, device="cuda") for _ in range(2))
        seq = torch.arange(B, dtype=torch.int32, device="cuda") * 9
        x, rows = start.clone(), []

        def done():
            if wait:
                torch.cuda.synchronize()

        binding.cache_append(None, *pre, kp, vp, front_table[None].contiguous(), ints([front]), cu_seqlens=ints([0, front]))
        done()
        for _ in range(steps):
            seq.add_(1)
            q = binding.cache_append(x, x[:, :Hkv], x[:, Hkv:2 * Hkv], kp, vp, table, seq, rope=rope)
            done()
            if shared:
                x = binding.decode_shared(q, kp, vp, front_table, ints([front]), table, seq)
            else:
                x = binding.decode_paged(q, kp, vp, table, seq)
            done()
            x = x + start * 0.5
            rows.append(x)
        torch.cuda.synchronize()
        return torch.stack(rows), kp, vp

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
