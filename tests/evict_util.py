"""Definitions of the drafted trees' and eviction's operators in 64 bits (plain Python where they are whole numbers),
and the error bounds of the computed ones.

Attention with any mask: the bound of paged_util.attend, whose derivation does not use the mask's form.

Weights.  out_j = decay w_j + sum_i p_ij, p_ij = exp(x_ij), x_ij = scale q_i.k_j - lse_i.  The kernel has, with e = 2^-24,
  q.k in fp32 from exact products: off by at most 2 d e sum |q k| (2: an accumulation that truncates), times |scale| in x
  scale and lse in log2 units, each rounded once, and one fma: e (|scale q.k| + |lse| + |x|)
  the exponential: 2^-22 relative
  the sum over n rows, all of one sign: at most n e relative, the four partial sums' joins in it
  the last fma: e |out|, and of the decayed old weight nothing else
so |out - exact| <= sum_i p_ij (|scale| 2 d e sum |q k| + e (|scale q.k| + |lse| + |x|) + 2^-22 + (n + 8) e) + e |out|, and 5%
for second order.  A p below 2^-126 may come out as 0: n 2^-126 more.
"""
import math

import torch

from tests.paged_util import U


def attend_seen(q, k, v, scale, seen, dtype):
    """q [n, Hq, d], k, v [L, Hkv, d] in float64, seen [n, L]: rows, log-sum-exp and error bound as paged_util.attend,
    and the log-sum-exp's: a sum of weights each off by u + e_s + 2^-21 relative, of which those of fp16 that vanish are 2^-32
    of the largest, a logarithm (2^-22) and a few roundings of values up to |lse| + 16 (in log2 units)."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    if L == 0:
        z = torch.zeros_like(q)
        return z, torch.full((n, Hq), -math.inf, device=q.device, dtype=q.dtype), z, z[..., 0]
    x = torch.einsum("nhgd,lhd->nhgl", q.view(n, Hkv, G, d), k) * scale
    size = torch.einsum("nhgd,lhd->nhgl", q.view(n, Hkv, G, d).abs(), k.abs()) * abs(scale)
    hidden = ~seen[:, None, None]
    x, size = x.masked_fill(hidden, -math.inf), size.masked_fill(hidden, 0.0)
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
    lse = (m + total.log()).squeeze(-1).reshape(n, Hq)
    off = 1.05 * (U[dtype] + e_s.reshape(n, Hq) + 2.0 ** -20 + L * 2.0 ** -32 + 2.0 ** -22 * (lse.abs() + 16))
    return o.reshape(n, Hq, d), lse, bound.reshape(n, Hq, d), off


def seen_of(mask, n, length):
    """[n, length] truth values of a sequence's n rows of mask words: the keys that each row sees."""
    words = mask.cpu().to(torch.int64) & 0xffffffff
    past = length - n
    seen = torch.zeros(n, length, dtype=torch.bool)
    if past > 0:
        seen[:, :past] = True
    for j in range(max(0, -past), n):
        seen[:, past + j] = (words[:, j // 32] >> (j % 32) & 1).bool()
    return seen.to(mask.device)


def mask_of(parents, words):
    """(mask rows, depths) of one tree, by walking up from every node."""
    rows, depth = [], []
    for i in range(len(parents)):
        bits, at, steps = 0, i, -1
        while at >= 0:
            bits |= 1 << at
            at, steps = parents[at], steps + 1
        row = [bits >> 32 * w & 0xffffffff for w in range(words)]
        rows.append([x - (1 << 32) if x >= 1 << 31 else x for x in row])
        depth.append(steps)
    return rows, depth


def weigh(q, k, lse, scale, seen):
    """Sums over rows for every key of one sequence, q [n, Hq, d], k [L, Hkv, d], lse [n, Hq] in float64, seen [n, L]:
    [Hkv, L] and their error bound."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    e = 2.0 ** -24
    out, bound = torch.zeros(2, Hkv, L, dtype=torch.float64, device=q.device)
    for h in range(Hkv):
        qh, kh, ls = q[:, h * G:(h + 1) * G], k[:, h], lse[:, h * G:(h + 1) * G, None]
        s = torch.einsum("ngd,ld->ngl", qh, kh) * scale
        size = torch.einsum("ngd,ld->ngl", qh.abs(), kh.abs()) * abs(scale)
        some = seen[:, None] & (ls > -math.inf)
        x = torch.where(some, s - ls, -math.inf)
        p = x.exp()
        off = 2 * d * e * size + e * (s.abs() + ls.abs() + (s - ls).abs()) + 2.0 ** -22 + (n * G + 8) * e
        out[h], bound[h] = p.sum((0, 1)), 1.05 * torch.where(some, p * off, 0.0).sum((0, 1)) + n * G * 2.0 ** -126
    return out, bound


def select(weights, n, budget, sink, recent):
    """The tokens of one row of n weights (a list) that stay, in rising order."""
    if n <= budget:
        return list(range(n))
    def rank(i):
        w = weights[i]
        return (0, 0.0, i) if math.isnan(w) else (1, -w, i)
    best = sorted(range(sink, n - recent), key=rank)[:budget - sink - recent]
    return sorted(list(range(sink)) + best + list(range(n - recent, n)))
