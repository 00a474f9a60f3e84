"""A model of how the paged-attention kernels cut their work (csrc/fa_paged.cuh), on the CPU.

Every CTA finds its own range of steps and walks its units without hearing of the others, and the join
reads the pieces from where the notes say they are.  Restated here over random batches: every unit's key
tiles are done once and in order, a CTA leaves at most one unit open (its last piece) and continues at
most one (its first), the note of an open unit names the CTA that closes it, and every CTA in between
holds exactly one piece of it.
"""
import random

import pytest


def tiles_of(seq, rb, rows, G, TK, causal):
    nq, length = seq
    seen = length
    if causal:
        seen = max(0, length - nq + min(nq - 1, (rb * rows + rows - 1) // G) + 1)
    return max(1, -(-seen // TK))


def units_of(seqs, Hkv, G, rows, TK, causal):
    """(sequence, kv head, block, tiles) in the order of the steps."""
    return [(b, hk, rb, tiles_of(s, rb, rows, G, TK, causal)) for b, s in enumerate(seqs) for hk in range(Hkv)
            for rb in range(-(-s[0] * G // rows))]


def both_of(seq, rb, rows, G, causal, tiles):
    """Key tiles of 128 that both query tiles of a block visit."""
    if rb * rows + rows // 2 >= seq[0] * G:
        return 0
    return min(tiles, tiles_of(seq, 2 * rb, rows // 2, G, 128, causal))


def weighted_pieces_of(units, unit_steps, both_steps, one_steps, grid):
    """pieces_of for units (sequence, head, block, tiles, both) whose key tiles cost both_steps for both query
    tiles (they come first) and one_steps for one: a range has the tiles that start in it."""
    def start(t, both, j):
        return unit_steps + min(j, both) * both_steps + max(0, j - both) * one_steps

    def starts_before(t, both, v):
        return sum(start(t, both, j) < v for j in range(t))

    W = sum(start(t, both, t) for *_, t, both in units)
    G = min(grid, max(W // both_steps, 1))
    ranges = [(c * W // G, (c + 1) * W // G) if c < G else (W, W) for c in range(grid)]
    out = [([], None) for _ in range(grid)]
    at = 0
    for i, (*_, t, both) in enumerate(units):
        cost = start(t, both, t)
        for c, (first, end) in enumerate(ranges):
            lo, hi = max(first, at), min(end, at + cost)
            if lo < hi:
                j0, j1 = starts_before(t, both, lo - at), starts_before(t, both, hi - at)
                if j1 > j0:
                    kind = 2 if j0 > 0 else (1 if j1 < t else 0)
                    out[c][0].append((i, j0, j1, kind))
                    if kind == 1:
                        out[c] = (out[c][0], cta_of(end + start(t, both, t - 1) - (hi - at), W, G))
        at += cost
    return out


def cta_of(step, W, G):
    c = min(((step + 1) * G - 1) // W, G - 1)
    while c > 0 and c * W // G > step:
        c -= 1
    while c + 1 < G and (c + 1) * W // G <= step:
        c += 1
    return c


def pieces_of(units, unit_steps, grid):
    """Per CTA: its pieces (unit, j0, j1, kind) and the CTA that closes the unit it leaves open, or None."""
    W = sum(t + unit_steps for *_, t in units)
    G = min(grid, max(W, 1))
    out = []
    for c in range(grid):
        first, end = (c * W // G, (c + 1) * W // G) if c < G else (W, W)
        pieces, at = [], 0
        for i, (*_, t) in enumerate(units):
            cost = t + unit_steps
            lo, hi = max(first, at), min(end, at + cost)
            if lo < hi:
                j0, j1 = max(0, lo - at - unit_steps), max(0, hi - at - unit_steps)
                if j1 > j0:
                    pieces.append((i, j0, j1, 2 if j0 > 0 else (1 if j1 < t else 0)))
            at += cost
        closes = None
        if pieces and pieces[-1][3] == 1:
            i, _, j1, _ = pieces[-1]
            closes = cta_of(end + (units[i][3] - j1) - 1, W, G)
        out.append((pieces, closes))
    return out


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_every_note_right(seed):
    rng = random.Random(seed)
    Hkv, G = rng.choice([1, 2, 8]), rng.choice([1, 3, 4, 7, 8, 16])
    tiled = rng.random() < 0.5
    rows, TK = (2 * (128 // G) * G, 128) if tiled else (rng.choice([16, 32, 64]), 64)
    seqs = [(rng.choice([0, 1, 1, rng.randint(1, 300)]), rng.choice([0, 1, rng.randint(1, 5000)]))
            for _ in range(rng.randint(1, 12))]
    units = units_of(seqs, Hkv, G, rows, TK, rng.random() < 0.6)
    grid = rng.choice([1, 2, 7, 152, 304])
    cut = pieces_of(units, rng.choice([0, 1, 2, 3]), grid)
    check_cut(units, cut)


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_when_tiles_cost_more_or_less(seed):
    rng = random.Random(2000 + seed)
    Hkv, G = rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 7, 16, 65, 100, 128])
    rows, causal = 2 * (128 // G) * G, rng.random() < 0.7
    seqs = [(rng.choice([0, 1, rng.randint(1, 300), rng.randint(1, 1200)]) // max(1, G // 16), rng.choice([0, 1, rng.randint(1, 3000)]))
            for _ in range(rng.randint(1, 6))]
    units = [(b, hk, rb, t, both_of(seqs[b], rb, rows, G, causal, t))
             for b, hk, rb, t in units_of(seqs, Hkv, G, rows, 128, causal)]
    both_steps, one_steps, unit_steps = rng.choice([(3, 2, 5), (3, 2, 5), (1, 1, 2), (4, 1, 0), (5, 5, 7)])
    grid = rng.choice([1, 2, 7, 40, 152])
    cut = weighted_pieces_of(units, unit_steps, both_steps, one_steps, grid)
    check_cut([u[:4] for u in units], cut)
    if (both_steps, one_steps) == (1, 1):
        assert cut == pieces_of([u[:4] for u in units], unit_steps, grid)


def check_cut(units, cut):
    done = {}
    for c, (pieces, closes) in enumerate(cut):
        for n, (i, j0, j1, kind) in enumerate(pieces):
            assert kind != 2 or n == 0
            assert kind != 1 or n == len(pieces) - 1
            done.setdefault(i, []).append((c, j0, j1, kind))
    assert sorted(done) == list(range(len(units)))
    for i, held in done.items():
        tiles = units[i][3]
        assert [h[1] for h in held] == [0] + [h[2] for h in held[:-1]] and held[-1][2] == tiles
        ctas = [h[0] for h in held]
        assert ctas == list(range(ctas[0], ctas[0] + len(held)))
        if len(held) == 1:
            assert held[0][3] == 0
        else:
            assert held[0][3] == 1 and all(h[3] == 2 for h in held[1:])
            assert cut[ctas[0]][1] == ctas[-1]


@pytest.mark.parametrize("seed", range(40))
def test_two_passes_split_the_sms(seed):
    """Both passes work out the same split from the same two sums: every SM is given once, each gets one at least."""
    rng = random.Random(1000 + seed)
    sms = rng.choice([2, 148, 152])
    mine, theirs = (rng.randint(1, 10 ** rng.randint(1, 12)) for _ in range(2))

    def share(is_first, own, other):
        first_ns = own if is_first else other
        first = min(max(sms * first_ns // (own + other), 1), max(sms - 1, 1))
        return first if is_first else max(sms - first, 1)

    a, b = share(True, mine, theirs), share(False, theirs, mine)
    assert a >= 1 and b >= 1 and a + b == sms
