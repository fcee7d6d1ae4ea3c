"""A NaN in one run of a context that a cluster shares reaches out and lse, however far the other runs' scores lie above."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("num_splits", [0, 1, 4])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("high", [100, -100, 0])
@pytest.mark.parametrize("at", [0, 5, 15])
def test_decode_scores_far_apart(at, high, d, num_splits):
    # 1024 tokens: a page of 64, every key of it NaN, is all that one of 16 CTAs has; one other page's scores are 800 or
    # -800 (or 0), the others' 0
    codes = torch.zeros((16, 2, 1, 64, d), dtype=torch.int8)
    codes[:, 1] = 50
    codes[7, 0] = high
    scales = torch.ones((16, 2, 1))
    scales[at, 0] = math.nan
    tables = torch.arange(16, dtype=torch.int32)[None].cuda()
    lse = torch.empty((1, 4), device="cuda")
    out = pkv.paged_attn_decode(codes.cuda(), torch.ones((1, 4, d)).half().cuda(), tables,
                                torch.tensor([1024], dtype=torch.int32).cuda(), scale=8.0 / d, lse=lse, num_splits=num_splits,
                                scales=scales.cuda())
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    # and without it the same call has numbers
    scales[at, 0] = 1.0
    out = pkv.paged_attn_decode(codes.cuda(), torch.ones((1, 4, d)).half().cuda(), tables,
                                torch.tensor([1024], dtype=torch.int32).cuda(), scale=8.0 / d, lse=lse, num_splits=num_splits,
                                scales=scales.cuda())
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
