"""A model of how kda_lin_fwd divides the chunks among its shares, and of the order in which the
state warps read initial states, publish and write final ones: with a state updated in place every
read of a unit's initial state has to come before the write of its final state, whatever the pace
of the shares.

The model repeats the kernel's rule (equal shares by weight in the order sequence, head, chunk; a unit
in two shares is handed over; a unit in more is summed before the main pass) and lists what each share
does in its program order.  Two actions of different shares are ordered only through a published
state or sum and the wait for it.  The model also carries what a state consists of, so a share that
starts from the wrong chunks is seen too.  Shares that read the initial state itself when they get to
a unit must fail (the planted mistake).
"""
import random

import pytest

C = 128


def share_starts(lens, heads, extra, ctas):
    """The units (sequence, head, chunks, weight before its chunks) and where, by weight, the shares start."""
    units, w = [], 0
    for n, length in enumerate(lens):
        for h in range(heads if length else 0):
            nc = (length + C - 1) // C
            units.append((n, h, nc, w + extra))
            w += nc + extra
    return units, [w * b // ctas for b in range(ctas + 1)]


def shares(lens, heads, extra, ctas):
    """For each share: the chunks of its sums, those of its main pass in order, how many of these it
    hands over, and how many come before the unit that the share before it began."""
    units, start = share_starts(lens, heads, extra, ctas)
    out = []
    for b in range(ctas):
        y0, y1 = start[b], start[b + 1]
        mine = [(u, c) for u, (_, _, nc, at) in enumerate(units) for c in range(nc) if y0 <= at + c < y1]
        sums, first, last = [], [], []
        if mine and mine[0][1] > 0:
            u = mine[0][0]
            _, _, nc, at = units[u]
            if at >= (start[b - 1] if b else 0) and at + nc <= y1:      # in two shares: taken last
                last = [m for m in mine if m[0] == u]
        if mine:
            u, c = mine[-1]
            _, _, nc, at = units[u]
            if c + 1 < nc:
                part = [m for m in mine if m[0] == u]
                if at >= y0 and at + nc <= start[min(b + 2, ctas)]:     # in two shares: taken first
                    first = part
                else:
                    sums = part
        middle = [m for m in mine if m not in first and m not in last]
        out.append((sums, first + middle + last, len(first), len(first) + len(middle)))
    return units, out


def actions(lens, heads, extra, ctas, kept):
    """Each share's actions in order: ("read" | "write" | "publish" | "wait" | "copied" | "begin", what).  `kept`: the
    share that begins a summed unit copies its initial state before it publishes its sum, and the unit's
    shares read the copy; else every share of the unit reads the state itself when it gets there."""
    units, div = shares(lens, heads, extra, ctas)
    acts = [[] for _ in range(ctas)]
    begins = {sums[0][0]: b for b, (sums, *_) in enumerate(div) if sums and sums[0][1] == 0} if kept else {}
    for b, (sums, main, n_first, n_before) in enumerate(div):
        if sums:
            u = sums[0][0]
            if begins.get(u) == b:
                acts[b].append(("read", u))
            acts[b].append(("publish", (u, frozenset(c for _, c in sums))))
        for i, (u, c) in enumerate(main):
            if i == 0 or main[i - 1] != (u, c - 1):
                before = []
                if c > 0 and i >= n_before:
                    before = [b - 1]
                elif c > 0:
                    before = [a for a in range(b) if div[a][0] and div[a][0][0][0] == u]
                acts[b] += [("wait", before)] if kept or i >= n_before else []
                if c == 0 or i < n_before:
                    acts[b].append(("copied", (u, begins[u])) if u in begins else ("read", u))
                acts[b] += [("wait", before), ("begin", (u, c))]
            if i + 1 == n_first:
                acts[b].append(("publish", (u, frozenset(range(c + 1)))))
            elif c + 1 == units[u][2]:
                acts[b].append(("write", u))
    return units, acts


def check(lens, heads, extra, ctas, kept=True):
    """The reads of an initial state that nothing orders before the write of the final one."""
    units, acts = actions(lens, heads, extra, ctas, kept)
    published = {b: (k, what) for b, a in enumerate(acts) for k, (kind, what) in enumerate(a) if kind == "publish"}
    assert len(published) == sum(kind == "publish" for a in acts for kind, _ in a), "a share publishes twice"
    # shares wait for lower ones only; seen[b][k][a]: how many actions of share a come before action k of
    # share b for certain
    seen = []
    for b, a in enumerate(acts):
        now, rows = {}, []
        for k, (kind, what) in enumerate(a):
            now = dict(now)
            now[b] = k + 1
            for w in what if kind == "wait" else []:
                assert w < b and w in published, f"share {b} waits for share {w}, which publishes nothing"
                for s, n in seen[w][published[w][0]].items():
                    now[s] = max(now.get(s, 0), n)
            rows.append(now)
        seen.append(rows)
    reads, writes = {u: [] for u in range(len(units))}, {u: [] for u in range(len(units))}
    for b, a in enumerate(acts):
        for k, (kind, what) in enumerate(a):
            if kind == "read":
                reads[what].append((b, k))
            elif kind == "write":
                writes[what].append((b, k))
            elif kind == "copied":      # the copy is the first action of the share that begins the unit
                u, w = what
                assert acts[w][0] == ("read", u) and seen[b][k].get(w, 0) > 0, f"share {b} reads a copy that may not be there"
            elif kind == "begin" and what[1] > 0:      # what the state holds when a later share begins
                sums = [published[w][1] for w in a[k - 1][1]]
                assert all(u == what[0] for u, _ in sums)
                assert frozenset().union(*(c for _, c in sums)) == frozenset(range(what[1])), (b, what)
    assert all(len(writes[u]) == 1 and reads[u] for u in reads)
    # copies are kept in slot share / 2: no two in one slot
    slots = [b // 2 for b, a in enumerate(acts) if len(a) > 1 and a[0][0] == "read" and a[1][0] == "publish" and a[1][1][0] == a[0][1]]
    assert not kept or len(set(slots)) == len(slots)
    return [(u, b) for u in reads for b, k in reads[u] if seen[writes[u][0][0]][writes[u][0][1]].get(b, 0) <= k]


BIG = [([8192], 32), ([8192], 64), ([32768], 32), ([4096], 40), ([12000], 40), ([16384], 64)]


@pytest.mark.parametrize("lens,heads", BIG, ids=[f"{'-'.join(map(str, a))}x{b}" for a, b in BIG])
@pytest.mark.parametrize("extra", [1, 2])
def test_initial_states_are_read_before_final_ones_are_written(lens, heads, extra):
    assert check(lens, heads, extra, 152) == []


@pytest.mark.parametrize("seed", range(40))
def test_initial_states_are_read_before_final_ones_are_written_drawn(seed):
    r = random.Random(seed)
    lens = [int(2 ** r.uniform(0, 12.5)) if r.random() < 0.9 else 0 for _ in range(r.randint(1, 6))] + [r.randint(1, 4000)]
    heads, ctas = r.choice([1, 2, 3, 7, 16, 30]), r.choice([1, 2, 3, 7, 40, 148, 152, 160])
    most = sum(n // C + 1 for n in lens) * heads
    assert check(lens, heads, r.choice([1, 2]), min(ctas, most)) == []


@pytest.mark.parametrize("lens,heads", [([8192], 32), ([32768], 32)])
def test_reading_the_initial_state_in_the_main_pass_is_too_late(lens, heads):
    assert check(lens, heads, 2, 152, kept=False)
