"""The few-token layer's ring, on the host: four fill warps (warp w takes the steps w,
w + 4, ...) wait for a stage's release by parity alone, which tells the release they
need from the one before but not from the one two before.  A model of the waits over
random schedules: with one thread issuing the MMAs, so that steps are released in
order, no step is filled before its stage is free; with two threads taking turns,
which may release a step before the one ahead of it, a five-stage ring is filled too
early."""

import random

import pytest

FILL_WARPS = 4


def run(stages, steps, issuers, rng):
    """-> whether some step was filled before the step `stages` before it was released."""
    released = [0] * stages                 # phases completed of a stage's release barrier
    filled, done = [False] * steps, [False] * steps
    at = list(range(FILL_WARPS))            # next step of each fill warp
    issue = list(range(issuers))            # next step of each MMA thread
    early = False
    while any(n < steps for n in issue):
        actors = [("fill", w) for w in range(FILL_WARPS) if at[w] < steps] + \
                 [("mma", i) for i in range(issuers) if issue[i] < steps]
        kind, i = rng.choice(actors)
        if kind == "fill":
            n = at[i]
            s, phase = n % stages, n // stages & 1
            if (released[s] & 1) != (phase ^ 1):            # try_wait(release, phase ^ 1)
                early |= n >= stages and not done[n - stages]
                filled[n] = True
                at[i] += FILL_WARPS
        else:
            n = issue[i]
            # its operands are there, and its partial buffer (of four) has been promoted,
            # which goes in order
            if filled[n] and all(done[:max(0, n - 3)]):
                done[n] = True
                released[n % stages] += 1
                issue[i] += issuers
    return early


@pytest.mark.parametrize("stages", [4, 5])
def test_one_issuer_never_too_early(stages):
    rng = random.Random(stages)
    assert not any(run(stages, rng.randint(1, 60), 1, rng) for _ in range(2000))


def test_two_issuers_break_the_five_stage_ring():
    rng = random.Random(7)
    assert any(run(5, 60, 2, rng) for _ in range(2000))
    assert not any(run(5, 9, 2, rng) for _ in range(2000))     # no stage is used a third time
    assert not any(run(4, 60, 2, rng) for _ in range(2000))    # a fill warp keeps its stage: it waited for each release
