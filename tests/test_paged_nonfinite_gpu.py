"""Attention over a paged cache with NaN and infinities in live queries, keys and values: a row comes out NaN where
the definition in 64 bits says so and right everywhere else, however the work is cut -- in clusters, in whole units,
in pieces that a join adds up, and in the two passes of a shared prefix."""
import math

import pytest
import torch

from attention_forward_prefill_gb300 import binding, build

from .paged_util import U, Cache, assert_rows

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    binding.load()
    binding.fa_device_status(True)
    yield
    assert binding.fa_device_status(True) == 0


def put(c, b, j, which, h, channel, value):
    """Key or value `which` ("k" or "v"), head h, of token j of sequence b (None: of the prefix), one channel of it."""
    table = c.prefix_table if b is None else c.table[b]
    (c.k if which == "k" else c.v)[int(table[j // c.page]), h, j % c.page, channel] = value
    (c.front if b is None else c.rows[b])[which == "v"][j, h, channel] = value


def expected(q, k, v, scale, causal, dtype):
    """attend() for rows that non-finite values reach: NaN where exp and sums give NaN.  A key whose score is -inf weighs
    nothing, as one that the mask hides."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    clean = lambda t: torch.where(t.isfinite(), t, 0.0)  # noqa: E731
    x = torch.einsum("nhgd,lhd->nhgl", q.view(n, Hkv, G, d), k) * scale
    size = torch.einsum("nhgd,lhd->nhgl", clean(q).view(n, Hkv, G, d).abs(), clean(k).abs()) * abs(scale)
    if causal:
        hidden = torch.arange(L, device=q.device) > L - n + torch.arange(n, device=q.device)[:, None]
        x = x.masked_fill(hidden[:, None, None], -INF)
    bad = (x.isnan() | (x == INF)).any(-1)
    x = x.masked_fill(bad[..., None], 0.0)
    size = size.masked_fill(x == -INF, 0.0)
    if L == 0:
        return torch.zeros_like(q), torch.full((n, Hq), -INF, device=q.device, dtype=q.dtype), torch.zeros_like(q)
    m = x.amax(-1, keepdim=True)
    e = torch.where(m == -INF, 0.0, (x - m).exp())
    total = e.sum(-1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0)
    o = torch.einsum("nhgl,lhd->nhgd", w, clean(v))
    # a value that is NaN reaches every row that sees its key, in its own channel
    nan = bad[..., None] | (torch.einsum("nhgl,lhd->nhgd", (x > -INF).double(), v.isnan().double()) > 0)
    # (the bound of attend)
    spread = torch.einsum("nhgl,lhd->nhgd", w, clean(v).abs()) + o.abs()
    bound = 1.05 * (U[dtype] + 2 * d * 2.0 ** -24 * size.amax(-1, keepdim=True) + 2.0 ** -21 + 2.0 ** -22 * 8) * spread
    if dtype == F16:
        bound = bound + L * 2.0 ** -32 * clean(v).abs().amax()
    lse = (m + total.log()).squeeze(-1).masked_fill(bad, NAN)
    return o.masked_fill(nan, NAN).reshape(n, Hq, d), lse.reshape(n, Hq), bound.reshape(n, Hq, d)


def check(got, want, bound, what):
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), f"{what}: {int((got.isnan() != nan).sum())} of {nan.numel()} NaN or not, wrongly"
    assert_rows(torch.where(nan, 0, got), torch.where(nan, 0.0, want), bound, what)


def rows_of(c, new, Hq, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(sum(new), Hq, c.d, generator=g, device="cuda").to(c.dtype)


def attention(c, q, new, causal, shared):
    """Rows and (of prefill_paged) their lse."""
    if shared:
        return binding.decode_shared(q, c.k, c.v, c.prefix_table, c.prefix_len, c.table, c.seq_lens), None
    if max(new) == 1:
        return binding.decode_paged(q, c.k, c.v, c.table, c.seq_lens), None
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32, device="cuda")
    lse = torch.empty(sum(new), q.shape[1], device="cuda")
    return binding.prefill_paged(q, c.k, c.v, c.table, c.seq_lens, cu, max(new), causal=causal, lse=lse), lse


# lens, new queries each, heads, head size, prefix, columns of the table behind the longest sequence
FORMS = {
    "cluster": ([300, 70, 0, 9], [1] * 4, 12, 4, 64, 0, 2),
    "cluster of one tile": ([30, 5], [1, 1], 4, 2, 128, 0, 2),
    "rows, cut": ([5000, 70, 0, 900], [1] * 4, 16, 2, 128, 0, 4000),
    "rows of 32, cut": ([3000, 70], [4, 3], 16, 2, 64, 0, 4000),
    "rows of 64, cut": ([3000, 70], [8, 3], 16, 2, 128, 0, 4000),
    "rows, whole": ([20 + i % 50 for i in range(700)], [1] * 700, 4, 2, 64, 0, 2),
    "tiles, cut": ([2500, 400], [300, 9], 4, 2, 128, 0, 2),
    "tiles of 64, cut": ([2500, 400], [300, 9], 4, 2, 64, 0, 2),
    "tiles, whole": ([140] * 160, [70] * 160, 2, 1, 128, 0, 2),
    "shared in clusters": ([0, 30, 70], [1] * 3, 12, 4, 64, 300, 2),
    "shared, two passes": ([0, 30, 700, 5] * 10, [1] * 40, 16, 2, 128, 3000, 4000),
    "shared, one row block": ([0, 30, 700, 5], [1] * 4, 8, 2, 64, 3000, 4000),
}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("what", ["query", "every key", "key", "infinite query", "infinite key", "value", "no score"])
def test_non_finite_rows(what, form, dtype):
    lens, new, Hq, Hkv, d, prefix, extra = FORMS[form]
    causal = max(new) > 1
    c = Cache(lens, Hkv, d, 16, dtype, seed=31, prefix=prefix, extra_cols=extra)
    q = rows_of(c, new, Hq, 7)
    if what == "query":  # one head of one token, in one channel
        q[0, 1, 3] = NAN
        q[-1, Hq - 1, d - 1] = NAN
    elif what == "infinite query":  # scores of +inf and -inf
        q[0, 1, 3] = INF
    elif what == "value":
        put(c, 0 if lens[0] else 1, 5, "v", 0, 11, NAN)
        if prefix:
            put(c, None, prefix - 1, "v", Hkv - 1, 2, NAN)
    else:
        spots = [(0, 0), (0, lens[0] // 2), (0, lens[0] - 1)] if lens[0] else [(1, lens[1] - 1)]
        if prefix:
            spots.append((None, prefix // 2))
        if what in ("every key", "no score"):  # of one head: a piece without one finite score
            for b in {b for b, _ in spots}:
                for j in range(prefix if b is None else lens[b]):
                    put(c, b, j, "k", 0, 0, NAN if what == "every key" else INF)
            if what == "no score":  # all -inf: as a row without keys
                q[:, :, 0] = -q[:, :, 0].abs().clamp(min=0.1)
        else:
            for b, j in spots:
                put(c, b, j, "k", 0, 0, NAN if what == "key" else INF)
            if what == "infinite key":
                # rows of one sign at the infinite channel: heads in turn see +inf and -inf
                sign = torch.where(torch.arange(Hq, device="cuda") % 2 == 0, 1.0, -1.0).to(dtype)
                q[:, :, 0] = q[:, :, 0].abs().clamp(min=0.1) * sign
    got, lse = attention(c, q, new, causal, prefix > 0)
    at = nans = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        k, v = c.keys(b)
        want, want_lse, bound = expected(q[at:at + n].double(), k, v, d ** -0.5, causal, dtype)
        check(got[at:at + n], want, bound, f"{what}, {form}, sequence {b}")
        nans += int(want.isnan().sum())
        if lse is not None:
            w = want_lse
            assert torch.equal(lse[at:at + n].isnan(), w.isnan())
            assert torch.equal(lse[at:at + n] == -INF, w == -INF)
            err = (lse[at:at + n].double() - w)[w.isfinite()].abs()
            assert err.numel() == 0 or err.max() <= 1.1 * 2.0 ** (-11 if dtype == F16 else -8) + 1e-4
        at += n
    assert (nans == 0) == (what == "no score")
    again, _ = attention(c, q, new, causal, prefix > 0)
    assert torch.equal(torch.nan_to_num(got, nan=77.0), torch.nan_to_num(again, nan=77.0))
