"""rope_frequencies where the ladder never gets down to the slow end of the blend: no GPU needed."""
import math

import pytest
import torch

from paged_kv_flash_cache_gb300 import rope


@pytest.mark.parametrize("rotary_dim,base,length,factor", [(128, 10000.0, 65536, 4.0), (128, 10000.0, 131072, 8.0),
                                                           (64, 10000.0, 1 << 20, 2.0), (128, 500000.0, 8192, 8.0),
                                                           (16, 10.0, 4096, 4.0), (64, 10000.0, 1 << 40, 16.0)])
def test_parts_blends_between_the_indices_of_fast_and_slow(rotary_dim, base, length, factor):
    """Each pair against the definition: kept up to the index (rounded down) of 32 turns over the trained context, divided by
    the factor from the index (rounded up, rotary_dim - 1 at most) of one turn, linear in the index between them."""
    half = rotary_dim // 2
    got, mscale = rope.rope_frequencies(rotary_dim, base, scaling="parts", factor=factor, original_length=length)
    assert mscale == pytest.approx(0.1 * math.log(factor) + 1)

    def index(turns):  # base^(-i / half) * length = 2 pi turns
        return half * math.log(length / (2 * math.pi * turns), base)
    low, high = max(math.floor(index(32)), 0), min(math.ceil(index(1)), rotary_dim - 1)
    for i in range(half):
        f = base ** (-i / half)
        if i <= low:
            want = f
        elif i >= high:
            want = f / factor
        else:
            t = (i - low) / (high - low)
            want = f * (1 - t) + f / factor * t
        assert float(got[i]) == pytest.approx(want, rel=1e-6), i


def test_parts_divides_no_pair_that_turns_more_than_slow():
    """128 elements, base 10000, trained on 65536 positions: the last pair makes 1.2 turns, so it is not yet divided in full."""
    got, _ = rope.rope_frequencies(128, 10000.0, scaling="parts", factor=4.0, original_length=65536)
    plain, _ = rope.rope_frequencies(128, 10000.0)
    ratio = (got / plain).double()
    turns = 65536 * plain.double() / (2 * math.pi)
    assert float(turns[-1]) > 1.19
    # indices 40 (of 32 turns, 40.2) and 65 (of one, 64.3): pair 63 is 23 / 25 of the way, pair 55 15 / 25
    assert float(ratio[-1]) == pytest.approx(1 - 0.75 * 23 / 25, abs=1e-6)
    assert float(ratio[55]) == pytest.approx(1 - 0.75 * 15 / 25, abs=1e-6)
    assert (ratio[turns > 1] > 0.25 + 1e-3).all() and (ratio.diff() <= 1e-6).all()


def test_parts_keeps_a_ladder_that_only_makes_fast_turns():
    got, _ = rope.rope_frequencies(64, 10000.0, scaling="parts", factor=16.0, original_length=1 << 62)
    plain, _ = rope.rope_frequencies(64, 10000.0)
    assert torch.equal(got, plain)
