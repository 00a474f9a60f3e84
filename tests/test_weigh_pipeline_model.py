"""The barrier protocol of the weighing on tensor-memory tiles, on the host (no GPU).

The roles of a CTA of weigh_tiles_kernel (csrc/fa_weigh_tiles_sm103.cu) -- the producer, the two product threads, the
warp of the log-sum-exps and the sixteen summing warps -- are restated as their waits, arrivals, loads and products, and
run under random interleavings: every run ends, no wait is overtaken by a phase, and every read finds what it expects.
Planted mistakes are caught.
"""
import random

import pytest

from tests.test_pipeline_model import ProtocolError, Sim

LOT = 4  # chunks of a lot of log-sum-exps


def weigh_kernel(sim, pieces, row_stages, plant=None):
    """pieces: for each piece with rows, its first and last (exclusive) chunk."""
    for i in range(4):
        sim.bar(f"k_full{i}")
        sim.bar(f"k_empty{i}")
    for i in range(row_stages):
        sim.bar(f"q_full{i}")
        sim.bar(f"q_empty{i}", 1 if plant == "a stage freed by one tile" else 2)
    for i in range(2):
        sim.bar(f"off_full{i}")
        sim.bar(f"off_empty{i}", 16)
        sim.bar(f"sum_full{i}", 4)
        sim.bar(f"sum_free{i}", 4)
        for odd in range(2):
            sim.bar(f"s_full{i}{odd}")
            sim.bar(f"s_free{i}{odd}", 4)

    def key_set(piece, t):
        return piece % 2 * 2 + t

    def producer():
        ch = 0
        for piece, (c0, c1) in enumerate(pieces):
            for t in range(2):
                s = key_set(piece, t)
                if piece >= 2 and plant != "keys loaded unasked":
                    yield "wait", f"k_empty{s}", piece // 2 - 1
                yield "load", [(f"K{s}", (piece, t))], f"k_full{s}"
            for c in range(c0, c1):
                qs = ch % row_stages
                if ch >= row_stages:
                    yield "wait", f"q_empty{qs}", ch // row_stages - 1
                yield "load", [(f"Q{qs}", (piece, c))], f"q_full{qs}"
                ch += 1

    def products(t):
        ch = 0
        for piece, (c0, c1) in enumerate(pieces):
            s = key_set(piece, t)
            yield "wait", f"k_full{s}", piece // 2
            for c in range(c0, c1):
                qs, buf = ch % row_stages, ch & 1
                if ch >= 2:
                    yield "wait", f"s_free{t}{buf}", ch // 2 - 1
                yield "wait", f"q_full{qs}", ch // row_stages
                yield ("mma", [(f"K{s}", (piece, t)), (f"Q{qs}", (piece, c))],
                       [(f"S{t}{buf}.{quad}", (piece, c)) for quad in range(4)])
                yield "commit", f"s_full{t}{buf}"
                yield "commit", f"q_empty{qs}"
                ch += 1
            yield "commit", f"k_empty{s}"

    def log_sum_exps():
        lots = 0
        for piece, (c0, c1) in enumerate(pieces):
            for c in range(c0, c1, LOT):
                os = lots % 2
                if lots >= 2:
                    yield "wait", f"off_empty{os}", lots // 2 - 1
                yield "write", f"off{os}", (piece, c)
                yield "arrive", f"off_full{os}"
                lots += 1

    def sums(t, odd, quad):
        ch = lots = several = 0
        for piece, (c0, c1) in enumerate(pieces):
            ch0 = ch
            for lot in range(c0, c1, LOT):
                os = lots % 2
                yield "wait", f"off_full{os}", lots // 2
                for c in range(lot, min(c1, lot + LOT)):
                    if ch & 1 == odd:
                        yield "wait", f"s_full{t}{odd}", ch // 2
                        if plant == "released before it is read" and quad == 2:
                            yield "arrive", f"s_free{t}{odd}"
                        yield "read", f"S{t}{odd}.{quad}", (piece, c)
                        yield "read", f"off{os}", (piece, lot)
                        if plant != "released before it is read" or quad != 2:
                            yield "arrive", f"s_free{t}{odd}"
                    ch += 1
                yield "arrive", f"off_empty{os}"
                lots += 1
            if c1 - c0 == 1:
                mine = ch0 & 1 == odd
            else:
                mine = not odd
                if odd:
                    if several and plant != "a sum handed over unasked":
                        yield "wait", f"sum_free{t}", several - 1
                    yield "write", f"sum{t}.{quad}", piece
                    yield "arrive", f"sum_full{t}"
                else:
                    yield "wait", f"sum_full{t}", several
                    yield "read", f"sum{t}.{quad}", piece
                    yield "arrive", f"sum_free{t}"
                several += 1
            if mine:
                yield "write", f"out{t}.{quad}.{piece}", "once" if sim.mem.get(f"out{t}.{quad}.{piece}") is None else "twice"

    sim.role("producer", producer())
    sim.role("log-sum-exps", log_sum_exps())
    for t in range(2):
        sim.role(f"products {t}", products(t))
        for odd in range(2):
            for quad in range(4):
                sim.role(f"sums {t}{odd}{quad}", sums(t, odd, quad))


def run(pieces, row_stages, seed, plant=None):
    sim = Sim(seed)
    weigh_kernel(sim, pieces, row_stages, plant)
    sim.run()
    for piece in range(len(pieces)):
        assert all(sim.mem[f"out{t}.{quad}.{piece}"] == "once" for t in range(2) for quad in range(4))


def some_pieces(rng):
    out = []
    for _ in range(rng.randint(1, 7)):
        c0 = rng.randint(0, 5)
        out.append((c0, c0 + rng.choice([1, 1, 2, 3, 4, 5, 9])))
    return out


@pytest.mark.parametrize("row_stages", [2, 8])
def test_the_protocol_holds(row_stages):
    rng = random.Random(row_stages)
    run([(0, 1)] * 8, row_stages, 1)
    run([(0, 2)] * 6, row_stages, 2)
    for seed in range(25):
        run(some_pieces(rng), row_stages, seed)


@pytest.mark.parametrize("plant", ["a stage freed by one tile", "keys loaded unasked", "released before it is read",
                                   "a sum handed over unasked"])
def test_planted_mistakes_are_caught(plant):
    caught = 0
    for seed in range(40):
        try:
            run([(0, 3), (0, 2), (1, 6), (0, 1), (0, 2), (0, 2)], 2, seed, plant)
        except ProtocolError:
            caught += 1
    assert caught
