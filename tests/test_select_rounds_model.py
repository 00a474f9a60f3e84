"""All exchanges of a selection's cluster, on the host (no GPU), from the first barrier to the last, and how it gives up.

tests/test_select_exchange_model.py has the rounds of one digit's counts and sums.  Here the threads of select_kernel
(csrc/fa_evict_sm103.cu), a group a CTA and part of the bins, also clear and fill the counts, arm the mbarriers (an arrival of
thread 0's that a phase needs besides what is sent), hand on what their tokens have, and give up when a wait runs out: every run
ends, reads find what they should, and nothing is sent to a CTA that has left.  Planted mistakes are caught.
"""
import random

import pytest

from tests.test_pipeline_model import ProtocolError, Sim

DIGITS = 3


class SlowStores(random.Random):
    """Leaves stores on their way for as long as others can go on, mostly."""

    def choice(self, choices):
        others = [c for c in choices if c[0] != "tma"]
        return super().choice(others if others and self.random() < 0.95 else choices)


class Cluster(Sim):
    """Stores that come in at a CTA whose groups have all left are a mistake; some of them get lost."""

    def __init__(self, seed, size, lost=0):
        super().__init__(seed)
        if seed % 2:
            self.rng = SlowStores(seed)
        self.size, self.lost = size, lost
        self.left = [0] * size

    def arrive(self, name):
        if name.startswith(("sent", "sums", "has")) and self.left[int(name.lstrip("senthasum"))] == self.size:
            raise ProtocolError(f"{name}: its CTA has left")
        super().arrive(name)

    def _ready(self, r):
        if r[2][0] == "landed":
            return not any(int(bar.lstrip("senthasum")) == r[2][1] for _, bar in self.tma)
        return super()._ready(r)

    def _step(self, r):
        if r[2][0] == "landed":
            return self._advance(r)
        if r[2][0] == "load" and self.rng.random() < self.lost:
            self._advance(r)  # (it never comes in)
        else:
            super()._step(r)


def exchange(sim, size, limit=None, plant=None):
    """limit: tests of a wait before it gives up, at most."""
    for c in range(size):
        sim.bar(f"sent{c}", size + 1)
        sim.bar(f"sums{c}", size + 1)
        sim.bar(f"has{c}", (size if plant == "every CTA expects all" else c) + 1)
        for b in ("counted", "read", "or", "found", "has_counted"):  # the CTA's own barriers
            sim.bar(f"cta_{b}{c}", size)
    sim.bar("cluster", size * size)
    ended = []

    def cta_barrier(name, c, digit):
        yield "arrive", f"cta_{name}{c}"
        yield "wait", f"cta_{name}{c}", digit

    def receive(bar, phase):
        if limit is None:
            yield "wait", bar, phase
            return True
        for _ in range(sim.rng.randint(1, limit)):
            if (yield "test", bar, phase):
                return True
        return False

    def leave(c):
        sim.left[c] += 1

    def give_up(c):
        if plant != "gives up without the cluster":
            yield "arrive", "cluster"
            yield "wait", "cluster", 1
        if plant != "gives up with stores on their way":
            yield "landed", c  # (the kernel waits for far longer than a store takes)
        leave(c)

    def group(c, g):  # of CTA c, the bins that CTA g adds up; the first holds thread 0
        if g == 0:
            for bar in ("sent", "sums", "has"):
                yield "arrive", f"{bar}{c}"
        yield "arrive", "cluster"
        for digit in range(DIGITS):
            for x in range(size):  # counts of this group's tokens
                yield "read", f"counts at {c} of {x} by {g}", ("clear", digit) if digit else None
                yield "write", f"counts at {c} of {x} by {g}", digit
            yield from cta_barrier("counted", c, digit)
            for by in range(size):
                yield "read", f"counts at {c} of {g} by {by}", digit
            if plant != "counts cleared late":
                for by in range(size):
                    yield "write", f"counts at {c} of {g} by {by}", ("clear", digit + 1)
            if digit == 0:
                yield "read", f"sums at {c} of {g}", None
                yield "wait", "cluster", 0  # all have started
            yield "load", [(f"sent to {g} by {c}", digit)], f"sent{g}"
            ok = yield from receive(f"sent{c}", digit)
            if g == 0 and ok and plant != "not armed again":
                yield "arrive", f"sent{c}"
            if ok:
                for r in range(size):
                    yield "read", f"sent to {c} by {r}", digit
            yield from cta_barrier("read", c, digit)
            if ok:
                yield "load", [(f"sums at {g} of {c}", digit)], f"sums{g}"
                if plant == "armed before it has come" and g == 0:
                    yield "arrive", f"sums{c}"
                ok = yield from receive(f"sums{c}", digit)
                if g == 0 and ok and plant != "armed before it has come":
                    yield "arrive", f"sums{c}"
                if ok:
                    yield "read", f"sums at {c} of {g}", digit
            if not ok:
                yield "write", f"failed {c} {g}", True
            yield from cta_barrier("or", c, digit)
            if any(sim.mem.get(f"failed {c} {x}") for x in range(size)):
                yield from give_up(c)
                return
            yield from cta_barrier("found", c, digit)
            if plant == "counts cleared late":
                for by in range(size):
                    yield "write", f"counts at {c} of {g} by {by}", ("clear", digit + 1)
        yield from cta_barrier("has_counted", c, 0)
        if g == 0:
            for r in range(c + 1, size):
                yield "load", [(f"has at {r} of {c}", "has")], f"has{r}"
        if plant != "has not waited for" and not (yield from receive(f"has{c}", 0)):
            yield from give_up(c)
            return
        for r in range(c):
            yield "read", f"has at {c} of {r}", "has"
        yield "arrive", "cluster"
        ended.append((c, g))
        yield "wait", "cluster", 1
        leave(c)

    for c in range(size):
        for g in range(size):
            sim.role(f"CTA {c} group {g}", group(c, g))
    return ended


def simulate(seed, size, limit=None, lost=0, plant=None):
    sim = Cluster(seed, size, lost)
    ended = exchange(sim, size, limit, plant)
    sim.run()
    assert sim.left == [size] * size  # all have left
    return len(ended)


@pytest.mark.parametrize("size", [2, 4, 8])
def test_the_rounds_hold(size):
    for seed in range(20):
        assert simulate(seed, size) == size * size


@pytest.mark.parametrize("size", [2, 4])
def test_all_leave_when_some_give_up(size):
    """Waits that run out too early, and stores that never come in: whoever goes on to the end has read what it should."""
    whole = 0
    for seed in range(60):
        whole += simulate(seed, size, limit=random.Random(seed).choice([3, 40, 2000])) == size * size
        assert simulate(seed, size, limit=60, lost=0.02) <= size * size
    assert 0 < whole < 60
    assert simulate(1, size, limit=60, lost=1) == 0


@pytest.mark.parametrize("plant,limit", [("not armed again", None), ("armed before it has come", None), ("every CTA expects all", None),
                                         ("counts cleared late", None), ("has not waited for", None), ("gives up without the cluster", 6),
                                         ("gives up with stores on their way", 6)])
def test_planted_mistakes_are_caught(plant, limit):
    caught = 0
    for seed in range(30):
        try:
            simulate(seed, 4, limit, plant=plant)
        except ProtocolError:
            caught += 1
    assert caught
