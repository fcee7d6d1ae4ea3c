"""The tcgen05 calls over an INT8 cache whose V scales are near FP32's smallest normal number, over contexts whose weights
add up to thousands: the scale over that sum has no normal number, the output has."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref
from tests.test_gpu_int8_decode import bounds, check, pool, tables_of

pytestmark = pytest.mark.gpu


def problem(lens, heads, d, scale, seed):
    bs = 16
    nb = sum(-(-n // bs) for n in lens) + 1
    codes, scales = pool(nb, heads, bs, d, seed)
    codes[:, 1] = codes[:, 1].abs() // 2 + 60                  # of one sign, so that nothing cancels
    scales[:, 1] = scale
    return codes, scales, tables_of(lens, bs, nb, max(-(-n // bs) for n in lens) + 1, seed)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -120, 2.0 ** -112])
@pytest.mark.parametrize("softmax_scale", [0.0, 0.02])
@pytest.mark.parametrize("num_splits", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
def test_many_heads(scale, softmax_scale, num_splits, d):
    lens = [2900, 300]
    codes, scales, tables = problem(lens, 1, d, scale, d)
    q = torch.randn((2, 20, d), generator=torch.Generator().manual_seed(1)).half()
    lse = torch.empty((2, 20), device="cuda")
    out = pkv.paged_attn_decode(codes.cuda(), q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                scale=softmax_scale, num_splits=num_splits, lse=lse, out_dtype=torch.float32, scales=scales.cuda())
    args = (codes.numpy(), scales.numpy(), q.double().numpy(), np.arange(3), lens, tables.numpy(), softmax_scale)
    ref, ref_lse = int8_ref.attention(*args, causal=False)
    err, err_lse = bounds(*args, ref, 2.0 ** -11, causal=False, weight_abs=2.0 ** -32)
    check(out, lse, ref, ref_lse, err + 16 * 2.0 ** -150, err_lse)  # (a merge's few sums near 2^-149)


@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -120, 2.0 ** -112])
@pytest.mark.parametrize("softmax_scale", [0.0, 0.02])
# a block of its own, blocks shared by a cluster, blocks of packed heads, blocks of enough sequences for a CTA each
@pytest.mark.parametrize("lens,new,hq,heads,d", [([2900, 260], [260, 200], 2, 2, 128), ([2900], [20], 4, 1, 64),
                                                 ([700] * 30, [140] * 30, 6, 6, 64)])
def test_prefill(lens, new, hq, heads, d, scale, softmax_scale):
    codes, scales, tables = problem(lens, heads, d, scale, d)
    cu = np.concatenate(([0], np.cumsum(new)))
    q = torch.randn((int(cu[-1]), hq, d), generator=torch.Generator().manual_seed(1)).half()
    lse = torch.empty(q.shape[:2], device="cuda")
    dev = [torch.tensor(np.asarray(x), dtype=torch.int32).cuda() for x in (cu, lens)]
    out = pkv.paged_attn_prefill(codes.cuda(), q.cuda(), dev[0], dev[1], tables.cuda(), max_q_len=max(new), scale=softmax_scale,
                                 lse=lse, out_dtype=torch.float32, scales=scales.cuda())
    args = (codes.numpy(), scales.numpy(), q.double().numpy(), cu, lens, tables.numpy(), softmax_scale)
    ref, ref_lse = int8_ref.attention(*args)
    err, err_lse = bounds(*args, ref, 2.0 ** -11, weight_abs=2.0 ** -32)
    check(out, lse, ref, ref_lse, err + 16 * 2.0 ** -150, err_lse)
