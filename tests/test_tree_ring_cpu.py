"""The ring of K and V tiles of paged_attn_tree over an FP8 cache, as the warps that convert the keys' codes see it.

They wait for the K tiles only. A barrier tells a waiter the parity of the phases that have completed, not their number: a
wait for phase p passes when an odd number of phases short of p have completed too. This model counts, for every K tile that they
come to, which loads can be outstanding, and checks that their waits do not pass before the tile has landed."""
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


def passes(landed, parity):
    """mbarrier.try_wait.parity: the phase in progress has the other parity."""
    return landed % 2 != parity


def early(segments, ring, waits):
    """K tiles whose waits can pass before they have landed."""
    items = ring_items(segments)
    found, last_k = [], None
    for k, kind in enumerate(items):
        if kind != "K":
            continue
        # what has landed for sure: the K tiles taken so far, and what the products had read before the last of them was sent for
        read = -1 if last_k is None else last_k - ring
        sure = [i for i in range(k) if items[i] == "K" or i <= read]
        maybe = [i for i in range(k) if i not in sure]                     # V tiles, in their order
        parity = (k // ring) % 2
        counts = [sum(1 for i in sure + maybe[:n] if i % ring == k % ring) for n in range(len(maybe) + 1)]
        # the waits one after the other, each with at least as many landed as the one before
        for at in itertools.combinations_with_replacement(range(len(counts)), len(waits)):
            if all(passes(counts[n], parity ^ w) for n, w in zip(at, waits)):
                found.append((k, at))
        last_k = k
    return found


CASES = [list(s) for n in (1, 2, 3, 4) for s in itertools.product([(True, 1), (True, 2), (True, 5), (False, 1), (False, 2), (False, 5)],
                                                                 repeat=n)]


@pytest.mark.parametrize("ring", [4, 5])
def test_the_conversion_waits_for_the_slots_last_tile_too(ring):
    for segments in CASES:
        if ring == 5 and any(wide for wide, _ in segments):
            continue                                                       # five slots: launches without wide blocks
        assert not early(segments, ring, waits=(1, 0)), segments


def test_one_wait_would_not_do():
    """A narrow segment's V tile on its way in the slot of the next, wide segment's first K."""
    assert early([(True, 5), (False, 5), (True, 5)], 4, waits=(0,))
