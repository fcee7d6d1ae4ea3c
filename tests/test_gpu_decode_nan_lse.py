"""A NaN in a query, or in one split's part of a context, over 16-bit and FP8 caches: NaN in out and lse, however many splits
the context has (a split's lse of -inf would take its part out of the merge, and the NaN with it)."""
from __future__ import annotations

import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# every decode kernel: groups of 1 and 2 (CUDA cores), 4 and 8 (mma.sync), others and head_dim 256 (tcgen05), FP8
@pytest.mark.parametrize("num_splits", [1, 5])
@pytest.mark.parametrize("hq,heads,d,fp8,dtype", [
    (2, 2, 128, False, "f16"), (4, 2, 64, False, "bf16"), (4, 1, 128, False, "bf16"), (8, 1, 64, False, "f16"),
    (3, 1, 128, False, "f16"), (32, 1, 128, False, "bf16"), (70, 1, 64, False, "f16"), (4, 2, 256, False, "bf16"),
    (2, 2, 128, True, "bf16"), (4, 1, 128, True, "f16"), (8, 1, 128, True, "bf16"), (16, 1, 128, True, "f16"), (4, 2, 64, True, "f16")])
def test_nan_of_a_sequence(hq, heads, d, fp8, dtype, num_splits):
    bs, n, batch = 16, 640, 4
    g = torch.Generator().manual_seed(hq + d)
    tables = torch.arange(batch * 40, dtype=torch.int32).reshape(batch, 40).cuda()
    shape = (batch * 40, 2, heads, bs, d)
    cache = torch.zeros(shape, dtype=torch.uint8 if fp8 else DT[dtype], device="cuda")
    scales = torch.zeros(shape[:4], device="cuda") if fp8 else None
    k, v = (torch.randn((batch * n, heads, d), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    pkv.kv_cache_append(cache, k, v, (torch.arange(batch + 1) * n).to(torch.int32).cuda(),
                        torch.zeros(batch, dtype=torch.int32).cuda(), tables, scales=scales)
    q = torch.randn((batch, hq, d), generator=g).to(DT[dtype]).cuda()
    lens = torch.tensor([n, n - 3, n, 130], dtype=torch.int32).cuda()

    def call():
        lse = torch.empty(q.shape[:2], device="cuda")
        return pkv.paged_attn_decode(cache, q, tables, lens, num_splits=num_splits, lse=lse, scales=scales), lse
    out, lse = call()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    q[0] = math.nan
    # sequence 2: one key of every head (with five splits: the second one's)
    page, row = int(tables[2, 10]), 7
    if fp8:
        scales[page, 0, :, row] = math.nan
    else:
        cache[page, 0, :, row, 3] = math.nan
    got, got_lse = call()
    for b in (0, 2):
        assert torch.isnan(got[b]).all() and torch.isnan(got_lse[b]).all(), b
    for b in (1, 3):
        assert torch.equal(got[b], out[b]) and torch.equal(got_lse[b], lse[b])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_combine_of_partials_with_a_nan(d):
    """Partial lse with NaN among numbers, alone, and behind 32 others; none, and all empty, as before."""
    g = torch.Generator().manual_seed(1)
    o, lse = torch.randn((5, 40, d), generator=g), torch.randn((5, 40), generator=g)
    lse[0, 3] = math.nan
    lse[1] = math.nan
    lse[2], lse[2, 39] = -math.inf, math.nan
    o[2, :39] = 0.0
    lse[3], o[3] = -math.inf, 0.0
    o[0, 3] = o[1] = o[2, 39] = math.nan
    got_lse = torch.empty(5, device="cuda")
    got = pkv.attn_combine(o.cuda(), lse.cuda(), lse=got_lse, out_dtype=torch.float32)
    assert torch.isnan(got[:3]).all() and torch.isnan(got_lse[:3]).all()
    assert got[3].eq(0).all() and got_lse[3].item() == -math.inf
    w = torch.softmax(lse[4].double(), 0)
    want = (w[:, None] * o[4].double()).sum(0)
    # 40 products and sums in FP32, exp to 2^-22
    assert (got[4].double().cpu() - want).abs().max() <= 48 * 2.0 ** -23 * (w[:, None] * o[4].double().abs()).sum(0).max() * 2
    assert abs(got_lse[4].item() - torch.logsumexp(lse[4].double(), 0).item()) <= 2.0 ** -20 * 4
