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
