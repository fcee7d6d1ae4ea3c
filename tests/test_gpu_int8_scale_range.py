"""How far V scales of one context may lie apart: powers of two down to 2^-24 of the largest are exact in the tcgen05 calls, and
down to 2^-35 of the largest of a tile in the decode of few heads."""
from __future__ import annotations

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv

pytestmark = pytest.mark.gpu


def mean_values(hq, d, below, new):
    """All weights equal (a softmax scale of 0), the large page's values 0: the mean of the small pages' values."""
    bs, n = 16, 200
    g = torch.Generator().manual_seed(d)
    codes = torch.randint(-127, 128, (13, 2, 1, bs, d), generator=g).to(torch.int8)
    scales = torch.full((13, 2, 1), below)
    codes[5, 1], scales[5] = 0, 1.0
    tables = torch.arange(13, dtype=torch.int32)[None].cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    args = dict(scale=0.0, out_dtype=torch.float32, scales=scales.cuda())
    if new:
        q = torch.zeros((new, hq, d)).half().cuda()
        out = pkv.paged_attn_prefill(codes.cuda(), q, torch.tensor([0, new], dtype=torch.int32).cuda(), lens, tables, max_q_len=new,
                                     causal=False, **args)
    else:
        out = pkv.paged_attn_decode(codes.cuda(), torch.zeros((1, hq, d)).half().cuda(), tables, lens, num_splits=1, **args)
    v = codes[:, 1, 0].reshape(-1, d)[:n].double()
    return out.double().cpu(), v.sum(0) / n * below, v.abs().sum(0) / n * below


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [0, 5, 200])
def test_exact_down_to_2_to_the_minus_24(d, new):
    for below in (2.0 ** -17, 2.0 ** -23, 2.0 ** -24):
        out, want, size = mean_values(16, d, below, new)
        # exact products of equal weights; FP32 sums of 200 (2^-23 a step at most) and the division
        assert torch.all((out - want).abs() <= 220 * 2.0 ** -23 * size), below


@pytest.mark.parametrize("d", [64, 128])
def test_few_heads_down_to_2_to_the_minus_30(d):
    # P' holds 2^-35 of the largest scale: of weights of 1, 2^-30 times them to 2^-36 2^30 = 2^-6 of a value at worst
    for below, eps in ((2.0 ** -17, 2.0 ** -19), (2.0 ** -24, 2.0 ** -12), (2.0 ** -30, 2.0 ** -6)):
        out, want, size = mean_values(4, d, below, 0)
        assert torch.all((out - want).abs() <= (220 * 2.0 ** -23 + eps) * size), below
