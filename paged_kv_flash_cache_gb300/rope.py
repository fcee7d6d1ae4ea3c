"""Rotary frequencies for `rope_append`: the plain geometric ladder and its scalings for contexts
longer than the ones a model was trained on. Host arithmetic in 64 bits, float32 result; nothing here
runs on the GPU.

The ladder: pair i of rotary_dim / 2 turns by base^(-2 i / rotary_dim) radians a position.
  linear   every frequency divided by `factor` (positions interpolated)
  ntk      the base grown to base * factor^(r / (r - 2)), r = rotary_dim: the lowest frequency is
           divided by factor, the highest is left alone
  parts    each frequency by the turns it makes over the trained context (`original_length`): those
           with at least `fast` turns are kept, those with at most `slow` are divided by factor, the
           ones between are blended linearly in the pair's index (between the indices at which the ladder, or
           its continuation, makes fast and slow turns, the second one rotary_dim - 1 at most); cosines and
           sines then carry 0.1 ln(factor) + 1
  smooth   the same two ends, blended linearly in the turns themselves; no factor on the cosines
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

SCALINGS = ("none", "linear", "ntk", "parts", "smooth")


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: Optional[int] = None, fast: Optional[float] = None,
                     slow: float = 1.0, device=None) -> Tuple["torch.Tensor", float]:
    """(inv_freq float32 [rotary_dim / 2], mscale) for `rope_append`. fast: 32 (parts) or 4 (smooth) if None."""
    import torch
    if rotary_dim <= 0 or rotary_dim % 16 != 0:
        raise ValueError("rotary_dim must be a positive multiple of 16")
    if scaling not in SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(SCALINGS))
    if not base > 1.0 or not factor >= 1.0 or not math.isfinite(base) or not math.isfinite(factor):
        raise ValueError("base > 1 and factor >= 1 required")
    if scaling in ("parts", "smooth") and (original_length is None or original_length <= 0):
        raise ValueError("%s scaling needs the trained context, original_length" % scaling)
    half = rotary_dim // 2
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = [base ** (-i / half) for i in range(half)]
    mscale = 1.0
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling in ("parts", "smooth"):
        fast = (32.0 if scaling == "parts" else 4.0) if fast is None else float(fast)
        if not fast > slow > 0:
            raise ValueError("fast > slow > 0 required")
        if scaling == "parts":
            # the index at which the ladder makes t turns over the trained context
            def index(t):
                return half * math.log(original_length / (2 * math.pi * t)) / math.log(base)
            low, high = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rotary_dim - 1)
            width = max(high - low, 1e-3)
            keep = [1.0 - min(max((i - low) / width, 0.0), 1.0) for i in range(half)]
            mscale = 0.1 * math.log(factor) + 1.0
        else:
            turns = [original_length * f / (2 * math.pi) for f in freq]
            keep = [min(max((t - slow) / (fast - slow), 0.0), 1.0) for t in turns]
        freq = [f * k + f / factor * (1.0 - k) for f, k in zip(freq, keep)]
    return torch.tensor(freq, dtype=torch.float64).to(torch.float32).to(device or "cpu"), mscale
