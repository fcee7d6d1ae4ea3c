"""The calls over an INT8 cache as a server makes them: prompts appended and attended to, sequences that continue them, decode
steps with new pages, pages that move to another pool; against the plain implementations, which follow the same host tables."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300.workloads import BlockAllocator
from tests import int8_ref
from tests.test_gpu_int8_decode import bounds, check

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def draw(g, n, heads, d):
    """Rows whose magnitudes differ by factors, so that pages' scales grow while sequences share what lies before."""
    x = torch.randn((n, heads, d), generator=g) * torch.exp2(torch.randn((n, heads, 1), generator=g))
    return x.bfloat16()


@pytest.mark.parametrize("hq", [4, 18])
def test_prompts_children_steps_and_another_pool(hq):
    heads, d, bs, nb, mb = 2, 128, 16, 64, 12
    g = torch.Generator().manual_seed(hq)
    scale = d ** -0.5
    pages = BlockAllocator(nb, bs, torch.randperm(nb, generator=g).tolist())
    codes = torch.randint(-127, 128, (nb, 2, heads, bs, d), generator=g, dtype=torch.int8)
    scales = torch.rand((nb, 2, heads), generator=g)
    gc, gs = codes.cuda(), scales.cuda()
    rc, rs = codes.numpy().copy(), scales.numpy().copy()

    def same():
        assert pkv.get_device_error() == 0
        assert np.array_equal(gs.cpu().numpy(), rs) and np.array_equal(gc.cpu().numpy(), rc)

    def near(out, lse, q, cu, lens, tables, causal, eps, small):
        args = (rc, rs, q.double().numpy(), cu, lens, tables, scale)
        ref, ref_lse = int8_ref.attention(*args, causal=causal)
        check(out, lse, ref, ref_lse, *bounds(*args, ref, eps, causal=causal, weight_abs=small))

    # ---- prompts ----
    lens = [37, 64, 5]
    tables = np.full((3, mb), -1, np.int32)
    for b, n in enumerate(lens):
        tables[b, :-(-n // bs)] = pages.allocate(n)
    cu = np.concatenate(([0], np.cumsum(lens)))
    k, v, q = draw(g, cu[-1], heads, d), draw(g, cu[-1], heads, d), draw(g, cu[-1], hq, d)
    pkv.kv_cache_append(gc, k.cuda(), v.cuda(), i32(cu), i32([0, 0, 0]), i32(tables), scales=gs)
    int8_ref.append(rc, rs, k.double().numpy(), v.double().numpy(), cu, [0, 0, 0], tables)
    same()
    lse = torch.empty((int(cu[-1]), hq), device="cuda")
    out = pkv.paged_attn_prefill(gc, q.cuda(), i32(cu), i32(lens), i32(tables), max_q_len=max(lens), lse=lse, scales=gs)
    near(out, lse, q, cu, lens, tables, True, 2.0 ** -11, 2.0 ** -32)

    # ---- children: three of the first prompt (one goes on in its page), two of the second, one of the third ----
    parents = [0, 0, 0, 1, 1, 2]
    fresh = [-1] + pages.allocate(5 * bs)
    t_dev, l_dev = pkv.kv_cache_fork(gc, i32(tables), i32(lens), i32(parents), i32(fresh), scales=gs)
    tables, lens = int8_ref.fork([(rc, 3), (rs, None)], tables, lens, parents, fresh, bs)
    same()
    assert np.array_equal(t_dev.cpu().numpy(), tables) and np.array_equal(l_dev.cpu().numpy(), lens)

    # ---- decode steps, a new page where one begins ----
    n = len(parents)
    for _ in range(20):
        for b in range(n):
            if tables[b, lens[b] // bs] < 0:
                tables[b, lens[b] // bs] = pages.allocate(1)[0]
        k, v, q = draw(g, n, heads, d), draw(g, n, heads, d), draw(g, n, hq, d)
        lse = torch.empty((n, hq), device="cuda")
        out = pkv.paged_attn_decode_step(gc, q.cuda(), i32(tables), i32(lens), k.cuda(), v.cuda(), lse=lse, scales=gs)
        eps, small = (2.0 ** -21, 2.0 ** -36) if hq <= 8 * heads else (2.0 ** -11, 2.0 ** -32)
        near(out, lse, q, np.arange(n + 1), lens, tables, False, eps, small)
        int8_ref.append(rc, rs, k.double().numpy(), v.double().numpy(), np.arange(n + 1), lens, tables)
        lens = lens + 1
        same()

    # ---- the last child's pages go to another pool: it reads the same there ----
    held = [int(p) for p in tables[-1][:-(-int(lens[-1]) // bs)]]
    there = torch.zeros((len(held) + 3, 2, heads, bs, d), dtype=torch.int8, device="cuda")
    there_scales = torch.zeros((len(held) + 3, 2, heads), device="cuda")
    to = list(range(len(held) + 1, 1, -1))
    pkv.kv_cache_copy(there, i32(held), i32(to), src_cache=gc, src_scales=gs, scales=there_scales)
    q = draw(g, 1, hq, d).cuda()
    here = pkv.paged_attn_decode(gc, q, i32(tables[-1:]), i32(lens[-1:]), scales=gs)
    table = np.full((1, mb), -1, np.int32)
    table[0, :len(to)] = to
    assert torch.equal(pkv.paged_attn_decode(there, q, i32(table), i32(lens[-1:]), scales=there_scales), here)
    assert pkv.get_device_error() == 0


def test_a_captured_round_and_a_second_stream():
    """Fork, step, copy in one graph, replayed, and the same calls on another stream while the graph runs on other pools: each
    leaves what the calls one by one leave."""
    heads, hq, d, bs, nb, mb = 2, 8, 64, 8, 40, 6
    g = torch.Generator().manual_seed(3)
    lens = [13, 29]
    tables = np.full((2, mb), -1, np.int32)
    tables[0, :2], tables[1, :4] = [3, 7], [11, 2, 30, 21]
    base = torch.randint(-127, 128, (nb, 2, heads, bs, d), generator=g, dtype=torch.int8).cuda()
    base_scales = torch.exp2(torch.randint(-8, -4, (nb, 2, heads), generator=g).float()).cuda()
    k, v, q = (draw(g, 4, h, d).cuda() for h in (heads, heads, hq))
    t, n, parents, fresh = i32(tables), i32(lens), i32([0, 1, 1, 0]), i32([5, 6, -1, 8])
    src, dst = i32([5, 6]), i32([39, 0])

    def calls(c, s, stream=None):
        ct, cn = pkv.kv_cache_fork(c, t, n, parents, fresh, scales=s, stream=stream)
        out = pkv.paged_attn_decode_step(c, q, ct, cn, k, v, scales=s, stream=stream)
        pkv.kv_cache_copy(c, src, dst, scales=s, stream=stream)
        return out

    pools = [(base.clone(), base_scales.clone()) for _ in range(3)]
    want = calls(*pools[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(*pools[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s in pools[1:]:
            c.copy_(base)
            s.copy_(base_scales)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        other = calls(*pools[2], stream=side)
        torch.cuda.synchronize()
        assert pkv.get_device_error() == 0
        assert torch.equal(out, want) and torch.equal(other, want)
        for c, s in pools[1:]:
            assert torch.equal(c, pools[0][0]) and torch.equal(s, pools[0][1])
