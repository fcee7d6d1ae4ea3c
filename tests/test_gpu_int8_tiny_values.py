"""paged_attn_decode over INT8 pages whose V scales lie at the lower end of their range: 2^11 over the largest scale of a tile
passes FP32's largest number there, and the scale over 2^11 its smallest normal one."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref
from tests.test_gpu_int8_decode import bounds, check, pool, tables_of

pytestmark = pytest.mark.gpu


def run(lens, scales_of, hq, heads, d, bs, num_splits, seed=3):
    """FP32 outputs within the bounds of the other sizes; a weight is 2^11 times itself relative to the power of two at or above
    its tile's largest scale, which may be twice that: 2^-35 for 2^-36. What a sum of numbers near FP32's smallest loses besides: half of
    2^-149 for each tile of a warp and each step of the merges, of a row whose weights add up to 1 at least."""
    nb = sum(-(-n // bs) for n in lens) + 1
    codes, scales = pool(nb, heads, bs, d, seed)
    mb = max(-(-n // bs) for n in lens) + 1
    tables = tables_of(lens, bs, nb, mb, seed)
    scales_of(scales, tables)
    q = torch.randn((len(lens), hq, d), generator=torch.Generator().manual_seed(seed)).half()
    lse = torch.empty((len(lens), hq), device="cuda")
    out = pkv.paged_attn_decode(codes.cuda(), q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), lse=lse,
                                num_splits=num_splits, out_dtype=torch.float32, scales=scales.cuda())
    assert pkv.get_device_error() == 0
    args = (codes.numpy(), scales.numpy(), q.double().numpy(), np.arange(len(lens) + 1), lens, tables.numpy(), d ** -0.5)
    ref, ref_lse = int8_ref.attention(*args, causal=False)
    err, err_lse = bounds(*args, ref, 2.0 ** -21, causal=False, weight_abs=2.0 ** -35)
    check(out, lse, ref, ref_lse, err + (max(lens) / 32 + 64) * 2.0 ** -150, err_lse)


# num_splits 0: few sequences, a cluster takes a context; 2: the splits and their merge
@pytest.mark.parametrize("num_splits", [0, 1, 2])
@pytest.mark.parametrize("d,heads,hq", [(64, 1, 1), (64, 2, 8), (128, 2, 4), (128, 1, 8)])
@pytest.mark.parametrize("scale", [2.0 ** -126, 1.37 * 2.0 ** -126, 2.0 ** -118, 2.0 ** -117, 1.9 * 2.0 ** -117, 2.0 ** -116,
                                   2.0 ** -115, 1.3 * 2.0 ** -115, 2.0 ** -114])
def test_every_page(scale, d, heads, hq, num_splits):
    def set_scales(scales, tables):
        scales[:, 1] = scale
    run([700, 33, 1], set_scales, hq, heads, d, 16, num_splits)


@pytest.mark.parametrize("num_splits", [0, 1, 2])
@pytest.mark.parametrize("d,heads,hq", [(64, 2, 4), (128, 1, 8)])
@pytest.mark.parametrize("scale", [2.0 ** -126, 1.37 * 2.0 ** -126, 2.0 ** -117])
def test_one_tile_among_others(scale, d, heads, hq, num_splits):
    """A page of 64 tokens (a tile or two) of tiny values among others, and one beside pages of zeros."""
    def set_scales(scales, tables):
        scales[tables[0, 4], 1] = scale
        scales[tables[1], 1] = 0.0
        scales[tables[1, 2], 1] = scale
    run([640, 300], set_scales, hq, heads, d, 64, num_splits)


@pytest.mark.parametrize("num_splits", [0, 1])
def test_appended_rows_of_tiny_values(num_splits):
    """As kv_cache_append writes bf16 rows of 2^-120: they come back as what was written, to half a step."""
    d, n = 128, 200
    g = torch.Generator().manual_seed(1)
    k = torch.randn((n, 1, d), generator=g).bfloat16()
    v = torch.full((n, 1, d), 1.5 * 2.0 ** -120).bfloat16()
    cache = torch.zeros((13, 2, 1, 16, d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((13, 2, 1), device="cuda")
    table = torch.arange(13, dtype=torch.int32)[None].cuda()
    pkv.kv_cache_append(cache, k.cuda(), v.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                        torch.zeros(1, dtype=torch.int32).cuda(), table, scales=scales)
    out = pkv.paged_attn_decode(cache, torch.randn((1, 4, d), generator=g).bfloat16().cuda(), table,
                                torch.tensor([n], dtype=torch.int32).cuda(), num_splits=num_splits, out_dtype=torch.float32,
                                scales=scales)
    # codes of 96 steps of 2^-126: exact, and a mean of equal values but for FP32's rounding (2^-21 of the weights' sum)
    assert (out / (1.5 * 2.0 ** -120) - 1).abs().max().item() < 2.0 ** -18
