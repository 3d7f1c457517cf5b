"""The activation backward's wind-down after a wait that ran out, on the host: a model
of its two stage barriers.  An item's copies are issued on stage n mod 2 once the item
two before has been read, and its wait is for parity (n / 2) mod 2.  Whatever item the
wait fails on, the wind-down's conditions hold only when no issued copy is in flight."""

import itertools

import pytest


class Barrier:
    """mbarrier with one arrival a phase: phases complete when their bytes land."""

    def __init__(self):
        self.done = 0          # phases completed

    def try_wait(self, parity):
        """True if the phase before the current one has this parity."""
        return (self.done & 1) != parity


def source_conditions():
    """The wind-down's `landed`, from the kernel's source."""
    import os
    with open(os.path.join(os.path.dirname(__file__), "..", "fp8_fine_grained_permute_b200", "csrc",
                           "act_backward.cu"), encoding="utf-8") as f:
        src = f.read()
    tail = src[src.index("void land_copies"):]
    return ("m >= items || mbar_try_wait(bars + 8u * (m & 1), (m >> 1) & 1)" in tail
            and "!(landed(n) && landed(n + 1))" in tail and "land_copies(full_bar(0), n, i1 - i0)" in tail)


@pytest.mark.parametrize("items", range(1, 8))
def test_no_copy_in_flight_when_the_cta_ends(items):
    assert source_conditions()
    for failed in range(items):
        # at the wait for item `failed`: items up to failed + 1 are issued, those
        # before it complete
        issued = [n for n in (failed, failed + 1) if n < items]
        for landed in itertools.product([False, True], repeat=len(issued)):
            bars = [Barrier(), Barrier()]
            for n in range(failed):
                bars[n & 1].done += 1
            for n, l in zip(issued, landed):
                bars[n & 1].done += l
            ends = all(n >= items or bars[n & 1].try_wait((n >> 1) & 1) for n in (failed, failed + 1))
            assert ends == all(landed), (failed, landed)
