"""Calls that allocate their outputs take every stream that CUDA has a handle for: the null, legacy and per-thread default streams
by number, a stream's own handle, and objects of other libraries that carry one."""
from __future__ import annotations

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv

pytestmark = pytest.mark.gpu


class Foreign:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("kind", ["f16", "int8"])
@pytest.mark.parametrize("which", ["0", "1", "2", "stream", "handle", "foreign", "foreign legacy", "default"])
def test_stream_handles(kind, which):
    side = torch.cuda.Stream()
    stream = {"0": 0, "1": 1, "2": 2, "stream": side, "handle": side.cuda_stream, "foreign": Foreign(side.cuda_stream),
              "foreign legacy": Foreign(1), "default": torch.cuda.default_stream()}[which]
    g = torch.Generator().manual_seed(1)
    cache, scales = torch.randn((12, 2, 2, 16, 128), generator=g).half().cuda(), None
    if kind == "int8":
        cache, scales = (cache.float() * 20).to(torch.int8), torch.full((12, 2, 2), 0.125, device="cuda")
    tables = torch.arange(12, dtype=torch.int32).reshape(1, 12).cuda()
    lens = torch.tensor([170], dtype=torch.int32).cuda()
    q = torch.randn((9, 4, 128), generator=g).half().cuda()
    cu, new = torch.tensor([0, 9], dtype=torch.int32).cuda(), torch.randn((1, 2, 128), generator=g).half().cuda()
    torch.cuda.synchronize()

    def calls(stream):
        yield pkv.paged_attn_decode(cache, q[:1], tables, lens, num_splits=2, stream=stream, scales=scales)
        yield pkv.paged_attn_decode_noalloc(cache, q[:1], tables, lens, stream=stream, scales=scales)
        yield pkv.paged_attn_prefill(cache, q, cu, lens, tables, max_q_len=9, stream=stream, scales=scales)
        yield pkv.paged_attn_mixed(cache, q, cu, lens, tables, max_q_len=9, stream=stream, scales=scales)
        yield from pkv.kv_cache_fork(cache, tables, lens, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                     torch.tensor([11, -1], dtype=torch.int32).cuda(), stream=stream, scales=scales)
        yield pkv.paged_attn_decode_step(cache, q[:1], tables, lens, new, new, stream=stream, scales=scales)
    want = [x.clone() for x in calls(None)]
    torch.cuda.synchronize()
    got = list(calls(stream))
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want) == 7
