"""A query row with a NaN, in a prefill over an INT8 cache: NaN in its output and in its lse (an lse of -inf would take the row
out of a later merge), whether a block is a CTA's or shared by a cluster; the other rows as without it."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_int8_decode import DT, pool, tables_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
# blocks of a CTA each, shared by clusters, of packed heads, of one tile
@pytest.mark.parametrize("lens,new,hq,heads,d", [([300] * 40, [200] * 40, 4, 4, 64), ([3000], [200], 2, 2, 128),
                                                 ([1500, 700], [20, 9], 8, 2, 64), ([130] * 60, [100] * 60, 3, 3, 128)])
def test_nan_in_a_query_row(lens, new, hq, heads, d, dtype):
    bs = 16
    nb = sum(-(-n // bs) for n in lens) + 1
    codes, scales = pool(nb, heads, bs, d, 2)
    tables = tables_of(lens, bs, nb, max(-(-n // bs) for n in lens) + 1, 2).cuda()
    cu = np.concatenate(([0], np.cumsum(new)))
    q = torch.randn((int(cu[-1]), hq, d), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    dev = [torch.tensor(np.asarray(x), dtype=torch.int32).cuda() for x in (cu, lens)]
    c, s = codes.cuda(), scales.cuda()

    def call(x):
        lse = torch.empty(q.shape[:2], device="cuda")
        return pkv.paged_attn_prefill(c, x, dev[0], dev[1], tables, max_q_len=max(new), lse=lse, scales=s), lse
    out, lse = call(q)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for row in (0, 5, int(cu[-1]) - 1):
        bad[row, row % hq] = True
    x = q.clone()
    x[bad] = math.nan
    got, got_lse = call(x)
    assert torch.isnan(got[bad]).all() and torch.isnan(got_lse[bad]).all()
    assert torch.equal(got[~bad], out[~bad]) and torch.equal(got_lse[~bad], lse[~bad])
