"""A workspace of decode_workspace_size bytes, the size that every format's documentation names, serves the decode and the mixed
call over an INT8 cache."""
from __future__ import annotations

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_int8_decode import pool

pytestmark = pytest.mark.gpu


def problem(batch, hq, heads, bs, mb, d=128):
    """Tables of any width over a few pages that all sequences share."""
    codes, scales = pool(4, heads, bs, d, 1)
    tables = torch.full((batch, mb), -1, dtype=torch.int32)
    tables[:, :min(4, mb)] = torch.arange(min(4, mb), dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(1, min(4, mb) * bs + 1, (batch,), generator=g, dtype=torch.int32)
    q = torch.randn((batch, hq, d), generator=g).half()
    return [x.cuda() for x in (codes, scales, tables, lens, q)]


# sizes where the splits that this decode would choose are smaller than those of the other formats
@pytest.mark.parametrize("batch,hq,heads,bs,mb", [(3, 32, 32, 256, 39), (227, 32, 8, 64, 9), (11, 32, 32, 16, 192),
                                                  (64, 32, 1, 16, 513), (16, 32, 32, 16, 513), (1, 32, 8, 16, 2000)])
def test_documented_size_is_enough(batch, hq, heads, bs, mb):
    codes, scales, tables, lens, q = problem(batch, hq, heads, bs, mb)
    need = pkv.decode_workspace_size(batch, hq, heads, 128, bs, mb)
    # with bytes behind it that no call may touch
    buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    want = pkv.paged_attn_decode(codes, q, tables, lens, scales=scales)
    got = pkv.paged_attn_decode(codes, q, tables, lens, scales=scales, workspace=buf[:need])
    cu = torch.arange(batch + 1, dtype=torch.int32).cuda()
    mixed = pkv.paged_attn_mixed(codes, q, cu, lens, tables, max_q_len=1, scales=scales, workspace=buf[:need])
    assert pkv.get_device_error() == 0
    assert torch.equal(got, want) and torch.equal(mixed, want)
    assert buf[need:].eq(77).all()
