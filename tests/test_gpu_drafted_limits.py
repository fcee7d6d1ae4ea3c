"""The drafted step's operators where sizes and places are unusual: pools whose offsets pass 32 bits, pages that sequences
share, many nodes and sequences, and over an FP8 cache the padded, empty and refused rows."""
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import rope
from paged_kv_flash_cache_gb300 import workloads as W
from tests.test_gpu_tree import Case
from tests.test_gpu_tree_fp8 import Fp8Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fp8", [False, True])
def test_a_pool_whose_offsets_pass_32_bits(fp8):
    """The whole step over pages at both ends of 4.7 * 10^9 cached elements: bit for bit what a small pool gives."""
    g = torch.Generator().manual_seed(1)
    hq, hkv, d, bs, far = 16, 8, 128, 64, 36000
    dt = torch.bfloat16
    ctx, n = [300, 130], [20, 40]
    pages = [[far - 1, 0, far - 2, 17, far - 9, far // 2], [far - 4, 1, far - 5, 2, 3, 4]]
    near = {p: i for i, p in enumerate(sorted(sum(pages, [])))}
    parents = [[-1] + [int(torch.randint(-1, i, (1,), generator=g)) for i in range(1, k)] for k in n]
    mask = W.tree_mask(parents).cuda()
    prompt, draft = (tuple(torch.randn((sum(t), h, d), generator=g).to(dt).cuda() for h in (hq, hkv, hkv)) for t in (ctx, n))
    inv, _ = rope.rope_frequencies(d, device="cuda")
    pos0 = torch.cat([torch.arange(c) for c in ctx]).to(torch.int32).cuda()
    depth = W.tree_depths(parents)
    pos1 = torch.cat([depth[:n[0]] + ctx[0], depth[n[0]:] + ctx[1]]).cuda()
    keep = [ctx[0] + i for i in (0, 3, 4, 19)] + [ctx[1] + i for i in (7, 9, 39)]

    def run(blocks, table):
        shape = (blocks, 2, hkv, bs, d)
        cache = torch.empty(shape, dtype=torch.uint8 if fp8 else dt, device="cuda")
        scales = torch.empty(shape[:4], device="cuda") if fp8 else None
        for p in sum(table, []):
            cache[p] = 0
            if fp8:
                scales[p] = 0
        t = i32(table)
        pkv.rope_append(cache, *prompt, inv, W.cu_lens(ctx).cuda(), i32([0, 0]), t, positions=pos0, scales=scales)
        q = pkv.rope_append(cache, *draft, inv, W.cu_lens(n).cuda(), i32(ctx), t, positions=pos1, scales=scales)
        out = pkv.paged_attn_tree(cache, q, mask, W.cu_lens(n).cuda(), i32([c + k for c, k in zip(ctx, n)]), t,
                                  max_q_len=max(n), scales=scales)
        pkv.kv_cache_compact(cache, i32(keep), i32([0, 4, 7]), i32(ctx), t, scales=scales)
        assert pkv.get_device_error() == 0
        rows = [cache[p].cpu() for p in sum(table, [])] + ([scales[p].cpu() for p in sum(table, [])] if fp8 else [])
        return q.cpu(), out.cpu(), rows

    small = run(len(near) + 1, [[near[p] for p in row] for row in pages])
    large = run(far, pages)
    assert torch.equal(small[0], large[0]) and torch.equal(small[1], large[1])
    assert all(torch.equal(a, b) for a, b in zip(small[2], large[2]))
    assert small[1].abs().max() > 0


def test_sequences_that_share_their_prefix_pages():
    c = Case([900, 900, 700], [9, 20, 3], 8, 2, bs=32, seed=3)
    c.table[1, :20] = c.table[0, :20]
    c.table[2, :15] = c.table[0, :15]
    c.check(c.run())


@pytest.mark.parametrize("make", [Case, Fp8Case])
def test_many_nodes_and_many_sequences(make):
    c = make([1500, 1001], [1000, 999], 4, 2, d=64, bs=16, seed=4, masks="any")
    c.check(c.run())
    g = torch.Generator().manual_seed(5)
    nodes = torch.randint(0, 4, (1500,), generator=g).tolist()
    lens = [max(1, k + int(torch.randint(0, 40, (1,), generator=g))) for k in nodes]
    c = make(lens, nodes, 2, 2, d=64, bs=8, seed=6, max_q=70)    # an upper bound well above the longest
    c.check(c.run())


def test_fp8_rows_that_see_nothing():
    for d in (64, 128):
        c = Fp8Case([20, 300], [20, 9], 8, 2, d=d, seed=5)
        for j in range(20):
            c.hide(0, 7, j)
            c.hide(0, 19, j)
        out, lse = c.run()
        c.check((out, lse))
        assert (out[7] == 0).all() and (lse[7] == -math.inf).all() and (lse[19] == -math.inf).all()


def test_fp8_padded_rows_bad_lengths_and_pages():
    c = Fp8Case([100, 60, 200], [5, 9, 4], 4, 2, seed=13)
    good, _ = c.run()
    codes, scales, table, cu = (t.cuda() for t in (c.codes, c.scales, c.table, c.cu))
    pad = 6
    q = torch.cat([c.q, torch.full((pad, 4, 128), math.nan, dtype=c.dt)]).cuda()
    mask = torch.cat([c.mask, torch.full((pad, c.mask.shape[1]), -1, dtype=torch.int32)]).cuda()

    def run(lens):
        out = torch.full(q.shape, 3.0, dtype=c.dt, device="cuda")
        pkv.paged_attn_tree(codes, q, mask, cu, i32(lens), table, max_q_len=9, out=out, scales=scales)
        code = pkv.get_device_error()
        assert (out[-pad:] == 3.0).all()
        return out[:-pad].cpu(), code

    out, code = run(c.lens)
    assert code == 0 and torch.equal(out, good)
    for lens in ([100, 8, 200], [100, table.shape[1] * c.bs + 1, 200], [100, -1, 200]):
        out, code = run(lens)
        assert code == 5 and (out[5:14] == 3.0).all()
        assert torch.equal(out[:5], good[:5]) and torch.equal(out[14:], good[14:])
    c.table[0, 2] = 10 ** 6
    c.run()
    assert pkv.get_device_error() == 5
    c.table[0, 2] = 0
    c.check(c.run())


def test_fp8_calls_repeat_on_streams_and_in_a_graph():
    c = Fp8Case([2500, 130], [30, 12], 8, 2, seed=17)
    want, _ = c.run()
    codes, scales, q, mask, cu, table = (t.cuda() for t in (c.codes, c.scales, c.q, c.mask, c.cu, c.table))
    lens = i32(c.lens)
    ws = [torch.full((pkv.tree_workspace_size(8, 2, 128, 30),), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, o in zip(side, ws, outs):
            pkv.paged_attn_tree(codes, q, mask, cu, lens, table, max_q_len=30, workspace=w, out=o, stream=s, scales=scales)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = pkv.paged_attn_tree(codes, q, mask, cu, lens, table, max_q_len=30, scales=scales)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.cpu(), want)
    assert pkv.get_device_error() == 0
