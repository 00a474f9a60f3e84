"""A paged cache with seeded contents, the definitions of the paged operators in 64 bits, one sequence
at a time, and the error bound of the attention over it.

Bound.  The kernels form S = q.k in fp32 from exact products, so a score is off by at most
e_s = 2 d 2^-24 sum |q_i k_i| |scale| (the factor 2 covers accumulation that truncates); ex2 adds 2^-21.
A weight is then rounded to the 16-bit type, off by u relative (2^-8 bf16, 2^-11 fp16), and the sum l adds
the rounded weights, so with w the exact weights
    |o - exact| <= (u + e_s + 2^-21) (sum w |v| + |exact|)
to first order; the rest below covers second order, fp32 sums, fp16 weights below the smallest step
(2^-32 of the largest, each key), and the output's own rounding.
"""
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class Cache:
    """Pages of K and V; sequence b owns the first ceil(lens[b] / page) entries of its table row."""

    def __init__(self, lens, Hkv, d, page, dtype, slots_first=False, seed=0, prefix=0, spare=2, extra_cols=2,
                 behind=float("nan"), total_pages=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // page) for n in lens]
        front = -(-prefix // page)
        used = sum(need) + front
        count = total_pages or used + spare
        shape = (count, page, Hkv, d) if slots_first else (count, Hkv, page, d)
        order = torch.randperm(count, generator=g, device="cuda")[:used] if total_pages is None else \
            torch.arange(count - used, count, device="cuda")
        raw = [torch.full(shape, behind, dtype=dtype, device="cuda") for _ in range(2)]
        self.k, self.v = (x.transpose(1, 2) if slots_first else x for x in raw)
        self.page, self.lens, self.prefix, self.Hkv, self.d, self.dtype = page, list(lens), prefix, Hkv, d, dtype
        cols = max(need + [0]) + extra_cols
        table, at = [], 0
        for n in need:
            table.append(order[at:at + n].tolist() + [-7] * (cols - n))
            at += n
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda").view(len(lens), cols)
        self.prefix_table = torch.tensor(order[at:at + front].tolist() + [-7], dtype=torch.int32, device="cuda")
        self.prefix_len = torch.tensor([prefix], dtype=torch.int32, device="cuda")
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        # real tokens
        self.rows, self.front = [], None
        for b, n in enumerate(lens):
            self.rows.append(self._fill(table[b], n, g))
        if prefix:
            self.front = self._fill(self.prefix_table.tolist(), prefix, g)

    def _fill(self, table, n, g):
        kv = torch.randn(2, n, self.Hkv, self.d, generator=g, device="cuda").to(self.dtype)
        if n:
            page = torch.tensor(table[:-(-n // self.page)], device="cuda").repeat_interleave(self.page)[:n]
            slot = torch.arange(n, device="cuda") % self.page
            self.k[page, :, slot], self.v[page, :, slot] = kv[0], kv[1]
        return kv[0].double(), kv[1].double()

    def keys(self, b):
        k, v = self.rows[b]
        if self.front is not None:
            k, v = torch.cat([self.front[0], k]), torch.cat([self.front[1], v])
        return k, v


def attend(q, k, v, scale, causal, dtype):
    """q [n, Hq, d], k, v [L, Hkv, d] in float64: rows, log-sum-exp and error bound (before the output's rounding)."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    x = torch.einsum("nhgd,lhd->nhgl", q.view(n, Hkv, G, d), k) * scale
    size = torch.einsum("nhgd,lhd->nhgl", q.view(n, Hkv, G, d).abs(), k.abs()) * abs(scale)
    if causal:
        i = torch.arange(n, device=q.device)[:, None]
        hidden = torch.arange(L, device=q.device) > L - n + i
        x = x.masked_fill(hidden[:, None, None], -math.inf)
        size = size.masked_fill(hidden[:, None, None], 0.0)
    if L == 0:
        z = torch.zeros_like(q)
        return z, torch.full((n, Hq), -math.inf, device=q.device, dtype=q.dtype), z
    m = x.amax(-1, keepdim=True)
    e = torch.where(m == -math.inf, 0.0, (x - m).exp())
    total = e.sum(-1, keepdim=True)
    w = torch.where(total > 0, e / total, 0.0)
    o = torch.einsum("nhgl,lhd->nhgd", w, v)
    spread = torch.einsum("nhgl,lhd->nhgd", w, v.abs()) + o.abs()
    e_s = 2 * d * 2.0 ** -24 * size.amax(-1, keepdim=True)
    bound = 1.05 * (U[dtype] + e_s + 2.0 ** -21 + 2.0 ** -22 * 8) * spread
    if dtype == torch.float16:
        bound = bound + L * 2.0 ** -32 * v.abs().amax()
    lse = (m + total.log()).squeeze(-1)
    return o.reshape(n, Hq, d), lse.reshape(n, Hq), bound.reshape(n, Hq, d)


def assert_rows(got, want, bound, what):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got.double() - want).abs()
    # the output's rounding, of a value that is itself within `bound` (a subnormal step at the least)
    tol = bound + U[got.dtype] * (want.abs() + bound) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    bad = err > tol
    if bad.any():
        at = torch.argmax(err - tol)
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} off; worst {got.flatten()[at].item()!r} for "
                             f"{want.flatten()[at].item()!r}, off {err.flatten()[at].item():.3e}, allowed "
                             f"{tol.flatten()[at].item():.3e}")
