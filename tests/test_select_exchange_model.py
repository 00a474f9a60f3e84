"""How the CTAs of a row's cluster exchange their counts in a selection, on the host (no GPU).

The threads of select_kernel (csrc/fa_evict_sm103.cu) that hold the bins of one part, a group a CTA and part, are restated
as their stores to other CTAs' shared memory, waits and reads, and run under random interleavings: every run ends, no wait
is overtaken by a phase, and every read finds this digit's counts or sums.  A planted mistake is caught.
"""
import random

import pytest

from tests.test_pipeline_model import ProtocolError, Sim

DIGITS = 3


class OneIsSlow(random.Random):
    """Leaves one role waiting for as long as others can go on, most of the time."""
    slow = None

    def choice(self, choices):
        others = [c for c in choices if not (c[0] == "role" and c[1][0] == self.slow)]
        return super().choice(others if others and self.random() < 0.999 else choices)


def simulate(seed, size, plant=None):
    sim = Sim(seed)
    sim.rng = OneIsSlow(seed)
    sim.rng.slow = f"CTA {seed % size} group {seed // size % size}" if seed % 3 else None
    exchange(sim, size, plant)
    sim.run()


def exchange(sim, size, plant=None):
    for c in range(size):
        sim.bar(f"sent{c}", size)
        sim.bar(f"sums{c}", size)
        for b in ("counted", "read", "found"):  # the CTA's own barriers
            sim.bar(f"{b}{c}", size)

    def cta_barrier(name, c, digit):
        yield "arrive", f"{name}{c}"
        yield "wait", f"{name}{c}", digit

    def group(c, g):  # of CTA c, the bins that CTA g adds up
        for digit in range(DIGITS):
            yield from cta_barrier("counted", c, digit)
            if digit == 0:
                yield "read", f"sums at {c} of {g}", None  # (counts of the first digit lie there too)
            yield "load", [(f"sent to {g} by {c}", digit)], f"sent{g}"
            yield "wait", f"sent{c}", digit
            for r in range(size):
                yield "read", f"sent to {c} by {r}", digit
            if plant != "sums sent before all have read":
                yield from cta_barrier("read", c, digit)
            yield "load", [(f"sums at {g} of {c}", digit)], f"sums{g}"
            yield "wait", f"sums{c}", digit
            yield "read", f"sums at {c} of {g}", digit
            yield from cta_barrier("found", c, digit)

    for c in range(size):
        for g in range(size):
            sim.role(f"CTA {c} group {g}", group(c, g))


@pytest.mark.parametrize("size", [2, 4, 8])
def test_the_exchange_holds(size):
    for seed in range(40):
        simulate(seed, size)


def test_a_planted_mistake_is_caught():
    """Sums that leave before all of the CTA's threads have read the counts: their receiver may be a digit ahead."""
    caught = 0
    for seed in range(40):
        try:
            simulate(seed, 4, "sums sent before all have read")
        except ProtocolError:
            caught += 1
    assert caught
