"""A query row with a NaN, in a prefill over a 16-bit or FP8 cache: NaN in its output and its lse (an lse of -inf would take the
row out of a later merge); the other rows as without it."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (256, False), (128, True)])
def test_nan_in_a_query_row(d, fp8, dtype):
    lens, new, hq, heads, bs = [300, 900, 40], [200, 300, 1], 4, 2, 16
    g = torch.Generator().manual_seed(d)
    need = [-(-n // bs) for n in lens]
    tables = torch.zeros((3, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    shape = (at, 2, heads, bs, d)
    tables = tables.cuda()
    cache = torch.zeros(shape, dtype=torch.uint8 if fp8 else DT[dtype], device="cuda")
    scales = torch.zeros(shape[:4], device="cuda") if fp8 else None
    cu_kv, cu = (torch.tensor(np.concatenate(([0], np.cumsum(x))), dtype=torch.int32).cuda() for x in (lens, new))
    k, v = (torch.randn((sum(lens), heads, d), generator=g).to(DT[dtype]).cuda() for _ in range(2))
    pkv.kv_cache_append(cache, k, v, cu_kv, torch.zeros(3, dtype=torch.int32).cuda(), tables, scales=scales)
    q = torch.randn((sum(new), hq, d), generator=g).to(DT[dtype]).cuda()
    n_lens = torch.tensor(lens, dtype=torch.int32).cuda()

    def call(x):
        lse = torch.empty(q.shape[:2], device="cuda")
        return pkv.paged_attn_prefill(cache, x, cu, n_lens, tables, max_q_len=max(new), lse=lse, scales=scales), lse
    out, lse = call(q)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for row in (0, 199, 350, 500):
        bad[row, row % hq] = True
    x = q.clone()
    x[bad] = math.nan
    got, got_lse = call(x)
    assert torch.isnan(got[bad]).all() and torch.isnan(got_lse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])
