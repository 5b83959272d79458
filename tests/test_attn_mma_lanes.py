"""A model of the 32 lanes of attention's MMA warp when bounded waits run out: each lane polls for itself
and comes to its own verdict, so some may give up at the very moment when others see the barrier
complete.  Whatever the verdicts, every lane has to reach the warp's end: what the whole warp does
together (a shuffle, a vote, a warp barrier) must not stand between lanes that have parted.

The lanes repeat the kernel's control flow: pieces of some blocks each, a vote and a first wait in front,
the waits of a block, the zeroed rows of a last block (an mbarrier of 32 arrivals with a bounded wait), a
vote behind.  The form with a plain break, a warp barrier and shuffles has to hang (the planted mistake).
"""
import random

import pytest

LANES = 32


def lane(pieces, verdict, together):
    """One lane: yields ("all", name, value) for what all lanes do together, ("zeros", n) for the bounded
    wait of the n-th zeroed tail.  verdict(): this lane's verdict of one wait."""
    zeros = 0
    for i, (blocks, tail) in enumerate(pieces):
        yield "all", "shuffle", True
        ok = yield "all", "vote", verdict()
        if ok:
            ok = verdict()
            if together:
                ok = yield "all", "vote", ok
        if not ok:
            break
        for j in range(blocks):
            ok = verdict()
            if ok and tail and j + 1 == blocks:
                if together:
                    ok = yield "zeros", zeros, None
                    zeros += 1
                else:
                    yield "all", "barrier", True
            if not ok or not (verdict() and verdict()):
                ok = False
                break
        if together:
            ok = yield "all", "vote", ok
        if not ok:
            break
    yield "all", "barrier", True


def run(seed, pieces, chance, together):
    """Whether every lane ends."""
    r = random.Random(seed)
    lanes = [lane(pieces, lambda: r.random() >= chance, together) for _ in range(LANES)]
    at = [next(x) for x in lanes]
    arrived = {}

    def step(k, value):
        try:
            at[k] = lanes[k].send(value)
        except StopIteration:
            at[k] = None

    while any(a is not None for a in at):
        waiting = [k for k in range(LANES) if at[k] is not None]
        for k in waiting:
            if at[k][0] == "zeros":
                arrived.setdefault(at[k][1], set()).add(k)
        done = [k for k in waiting if at[k][0] == "zeros" and len(arrived[at[k][1]]) == LANES]
        if not done and len(waiting) == LANES and all(at[k][:2] == at[0][:2] and at[k][0] == "all" for k in waiting):
            value = all(at[k][2] for k in waiting)
            for k in waiting:
                step(k, value)
            continue
        if done:
            for k in done:
                step(k, True)
            continue
        late = [k for k in waiting if at[k][0] == "zeros"]      # their limit runs out
        if not late:
            return False
        for k in late:
            step(k, False)
    return True


PIECES = [[(3, True)], [(1, True), (4, False), (2, True)], [(5, False)] * 3, [(1, True)] * 4]


@pytest.mark.parametrize("chance", [0.0, 0.002, 0.02, 0.5])
@pytest.mark.parametrize("pieces", PIECES, ids=range(len(PIECES)))
def test_every_lane_reaches_the_end(pieces, chance):
    assert all(run(seed, pieces, chance, True) for seed in range(100))


@pytest.mark.parametrize("pieces", PIECES[1:], ids=range(1, len(PIECES)))
def test_lanes_that_part_before_an_exchange_hang(pieces):
    assert not all(run(seed, pieces, 0.002, False) for seed in range(100))
