"""The no-allocation decode over an INT8 cache: its array serves every call that needs no more than that, by this format's own
splits, however much the other formats' would need."""
from __future__ import annotations

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_int8_workspace import problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,hq,heads,bs,mb", [(4, 128, 1, 16, 2048), (8, 64, 1, 16, 1024)])
def test_no_allocation_where_the_other_formats_need_more(batch, hq, heads, bs, mb):
    codes, scales, tables, lens, q = problem(batch, hq, heads, bs, mb)
    limit = pkv.DECODE_NOALLOC_SCRATCH_BYTES
    assert pkv.decode_workspace_size(batch, hq, heads, 128, bs, mb) > limit
    want = pkv.paged_attn_decode(codes, q, tables, lens, scales=scales)
    got = pkv.paged_attn_decode_noalloc(codes, q, tables, lens, scales=scales)
    assert pkv.get_device_error() == 0 and torch.equal(got, want)


def test_no_allocation_refuses_what_does_not_fit():
    codes, scales, tables, lens, q = problem(64, 32, 8, 16, 2048)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attn_decode_noalloc(codes, q, tables, lens, scales=scales)
