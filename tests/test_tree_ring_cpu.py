"""The ring of K and V tiles of paged_attn_tree over an FP8 cache, as the warps that convert the keys' codes see it.

They take the K tiles only. A barrier tells a waiter the parity of the phases that have completed, not their number: a wait for phase
p passes when an odd number of phases short of p have completed too, and holds again once phase p + 1 has. This model goes, for
every K tile that they come to, through all that can have been loaded and read by then, and checks that their waits neither pass
before the tile has landed nor hold for good."""
from __future__ import annotations

import itertools

import pytest


def ring_items(segments):
    """The ring's order of use: K of the first `ahead` tiles, then V_j, K_(j + ahead), and the last V's."""
    items = []
    for wide, tiles in segments:
        ahead = 1 if wide else min(2, tiles)
        items += ["K"] * ahead
        for j in range(tiles):
            items.append("V")
            if j + ahead < tiles:
                items.append("K")
    return items


def passes(done, parity):
    """mbarrier.try_wait.parity: the phase in progress has the other parity."""
    return done % 2 != parity


def states(items, ring, k, last_k):
    """(items read, set of items landed) that are possible while the warps are at K tile k, having taken last_k before.

    The products read the items in order, each after it has landed (a K tile: after it was converted, so none from k on); an
    item is sent for once the one before it in its slot has been read, and lands any time after that."""
    read_min = 0 if last_k is None else max(0, last_k - ring + 1)          # last_k was sent for: items up to last_k - ring are read
    for read in range(read_min, k + 1):
        sent = range(min(len(items), read + ring))
        sure = {i for i in sent if i < read or (items[i] == "K" and i < k)}
        maybe = [i for i in sent if i not in sure]
        for n in range(1 << len(maybe)):
            yield read, sure | {i for b, i in enumerate(maybe) if n >> b & 1}


def count(done, k, ring):
    return sum(1 for i in done if i % ring == k % ring)


def faults(segments, ring, waits):
    """(K tiles whose waits can pass before they have landed, K tiles at which they can hold for good). `waits`: (barrier, flip)."""
    items = ring_items(segments)
    early, stuck, last_k = [], [], None
    for k, kind in enumerate(items):
        if kind != "K":
            continue
        parity = (k // ring) % 2
        seen = list(states(items, ring, k, last_k))

        def ok(state, wait):
            bar, flip = wait
            read, landed = state
            return passes(count(landed if bar == "full" else range(read), k, ring), parity ^ flip)

        # the waits one after the other, in states that follow one another
        at = [s for s in seen if ok(s, waits[0])]
        for wait in waits[1:]:
            at = [t for t in seen if ok(t, wait) and any(s[0] <= t[0] and s[1] <= t[1] for s in at)]
        if any(k not in landed for _, landed in at):
            early.append(k)
        # when everything before k is read and all that was sent for has landed, nothing more happens without these warps
        final = (k, set(range(min(len(items), k + ring))))
        if not all(ok(final, w) for w in waits):
            stuck.append(k)
        last_k = k
    return early, stuck


SEGMENTS = [(True, 1), (True, 2), (True, 5), (False, 1), (False, 2), (False, 3), (False, 5)]
CASES = [list(s) for n in (1, 2, 3) for s in itertools.product(SEGMENTS, repeat=n)]
CASES += [[(True, 5), (False, 5), (True, 5), (False, 2)], [(False, 1)] * 9, [(True, 1)] * 9]


@pytest.mark.parametrize("ring", [4, 5])
def test_read_then_landed(ring):
    """The slot's last tile read, then this one landed: what the warps wait for."""
    for segments in CASES:
        if ring == 5 and any(wide for wide, _ in segments):
            continue                                                       # five slots: launches without wide blocks
        assert faults(segments, ring, (("empty", 1), ("full", 0))) == ([], []), segments


def test_landed_alone_passes_early():
    """A narrow segment's V tile on its way in the slot of the next, wide segment's first K."""
    assert faults([(True, 5), (False, 5), (True, 5)], 4, (("full", 0),))[0]


def test_landed_twice_can_hold_for_good():
    """kv_full for the slot's last tile, then for this one: the first holds once this one has landed."""
    assert faults([(True, 5)], 4, (("full", 1), ("full", 0)))[1]
