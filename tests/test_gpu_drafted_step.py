"""A drafted decoding step as it is used: rope_append writes the drafted tokens' rows (rotary position = context +
depth, slot = context + node), paged_attn_tree verifies the tree, kv_cache_compact keeps the accepted path. What is left has
to be the cache that the accepted tokens would have built one after the other."""
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import rope
from paged_kv_flash_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def path_to(parents, node):
    out = []
    while node >= 0:
        out.append(node)
        node = parents[node]
    return out[::-1]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 2, 128, 16), (4, 4, 64, 8), (16, 2, 128, 32)])
def test_accepted_path_leaves_the_sequential_cache(hq, hkv, d, bs, fp8):
    g = torch.Generator().manual_seed(hq + d + bs)
    dt = torch.bfloat16
    ctx = [37, 5, 300]
    parents = [[-1, 0, 0, 1, 1, 3, 2], [-1, -1, 1, 2, 3], [-1] + list(range(12))]
    accepted = [5, 4, 12]            # the node whose path is accepted
    n = [len(p) for p in parents]
    batch = len(ctx)
    need = [-(-(c + k) // bs) for c, k in zip(ctx, n)]
    alloc = W.BlockAllocator(sum(need) + 3, bs, torch.randperm(sum(need) + 3, generator=g).tolist())
    table = W.block_table_tensor([alloc.allocate(c + k) for c, k in zip(ctx, n)], max(need)).cuda()
    shape = (sum(need) + 3, 2, hkv, bs, d)
    inv, mscale = rope.rope_frequencies(d, 10000.0, scaling="parts", factor=4.0, original_length=64, device="cuda")
    qw, kw = (1 + 0.1 * torch.randn((2, d), generator=g)).to(dt).cuda()

    def empty():
        if fp8:
            return torch.zeros(shape, dtype=torch.uint8, device="cuda"), torch.zeros(shape[:4], device="cuda")
        return torch.zeros(shape, dtype=dt, device="cuda"), None

    def rows(count):
        return torch.randn((count, (hq + 2 * hkv) * d), generator=g).to(dt).cuda()

    def append(cache, scales, x, new, before, positions):
        q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
        return pkv.rope_append(cache, q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d)), inv,
                               W.cu_lens(new).cuda(), i32(before), table, positions=positions, mscale=mscale, q_weight=qw,
                               k_weight=kw, scales=scales)

    prompt, draft = rows(sum(ctx)), rows(sum(n))
    cache, scales = empty()
    prompt_pos = torch.cat([torch.arange(c) for c in ctx]).to(torch.int32).cuda()
    append(cache, scales, prompt, ctx, [0] * batch, prompt_pos)
    base, base_scales = cache.clone(), None if scales is None else scales.clone()
    depth = W.tree_depths(parents)
    pos = torch.cat([depth[sum(n[:b]):sum(n[:b + 1])] + ctx[b] for b in range(batch)]).cuda()
    q = append(cache, scales, draft, n, ctx, pos)

    paths = [path_to(p, a) for p, a in zip(parents, accepted)]
    start = [sum(n[:b]) for b in range(batch)]
    mask = W.tree_mask(parents).cuda()
    out = pkv.paged_attn_tree(cache, q, mask, W.cu_lens(n).cuda(), i32([c + k for c, k in zip(ctx, n)]), table,
                              max_q_len=max(n), out_dtype=torch.float32, scales=scales)

    # the accepted path moves to the front of the drafted rows, whose pages' other rows stay the draft's
    keep = [ctx[b] + i for b in range(batch) for i in paths[b]]
    pkv.kv_cache_compact(cache, i32(keep), W.cu_lens([len(p) for p in paths]).cuda(), i32(ctx), table, scales=scales)
    assert pkv.get_device_error() == 0

    # the same tokens one after the other
    seq, seq_scales = base, base_scales
    longest = max(len(p) for p in paths)
    for step in range(longest):
        live = [b for b in range(batch) if step < len(paths[b])]
        new = [1 if b in live else 0 for b in range(batch)]
        x = torch.stack([draft[start[b] + paths[b][step]] for b in live])
        qs = append(seq, seq_scales, x, new, [ctx[b] + step for b in range(batch)], i32([ctx[b] + step for b in live]))
        # each step's query attends to what is cached by then: the tree's row of that node
        lens = i32([ctx[b] + step + 1 for b in live])
        ref = pkv.paged_attn_decode(seq, qs, table[live].contiguous(), lens, out_dtype=torch.float32, scales=seq_scales)
        for i, b in enumerate(live):
            got = out[start[b] + paths[b][step]]
            # both sides sum in FP32: the score's 0.9 D^1.5 2^-24 and P's 2^-17, twice each, of max|v| < 6; over an FP8 cache
            # the tree's values are rounded to bf16 (half a step, 2^-8) and the decode's weights to f16 (2^-11)
            tol = 4 * (0.9 * d ** 1.5 * 2.0 ** -24 + 2.0 ** -17) + (2.0 ** -8 + 2.0 ** -10 if fp8 else 0.0)
            assert (got - ref[i]).abs().max() <= tol * 6
    for b in range(batch):
        for p in range(ctx[b] + len(paths[b])):
            pg, off = int(table[b, p // bs]), p % bs
            assert torch.equal(cache[pg, :, :, off], seq[pg, :, :, off]), (b, p)
            if fp8:
                assert torch.equal(scales[pg, :, :, off], seq_scales[pg, :, :, off])
    # and the next step over either cache is the same
    lens = i32([ctx[b] + len(paths[b]) for b in range(batch)])
    q1 = torch.randn((batch, hq, d), generator=g).to(dt).cuda()
    a = pkv.paged_attn_decode(cache, q1, table, lens, scales=scales)
    b_ = pkv.paged_attn_decode(seq, q1, table, lens, scales=seq_scales)
    assert torch.equal(a, b_)
    assert pkv.get_device_error() == 0


def test_whole_step_in_one_graph():
    """append, verify and compact captured together and replayed over new drafts."""
    g = torch.Generator().manual_seed(4)
    hq, hkv, d, bs, n, ctx = 8, 2, 128, 16, 8, 100
    dt = torch.float16
    nb = -(-(ctx + n) // bs)
    table = torch.randperm(nb, generator=g).to(torch.int32)[None].cuda()
    cache = torch.randn((nb, 2, hkv, bs, d), generator=g).to(dt).cuda()
    first = cache.clone()
    inv, _ = rope.rope_frequencies(d, device="cuda")
    parents = [[-1, 0, 0, 1, 1, 2, 2, 3]]
    mask, depth = W.tree_mask(parents).cuda(), (W.tree_depths(parents) + ctx).cuda()
    q, k, v = (torch.zeros((n, h, d), dtype=dt, device="cuda") for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    cu, before, lens = i32([0, n]), i32([ctx]), i32([ctx + n])
    keep, cu_keep = i32([ctx, ctx + 1, ctx + 4, 0]), i32([0, 3])
    ws = torch.empty(pkv.tree_workspace_size(hq, hkv, d, n), dtype=torch.uint8, device="cuda")

    def step():
        qr = pkv.rope_append(cache, q, k, v, inv, cu, before, table, positions=depth)
        pkv.paged_attn_tree(cache, qr, mask, cu, lens, table, max_q_len=n, workspace=ws, out=out)
        pkv.kv_cache_compact(cache, keep, cu_keep, before, table)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(dt))
        cache.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        got, kept = out.clone(), cache.clone()
        cache.copy_(first)
        step()
        torch.cuda.synchronize()
        assert torch.equal(out, got) and torch.equal(cache, kept)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("as_handle", [False, True])
def test_new_tensors_belong_to_the_calls_stream(as_handle):
    """With a `stream` of the caller's, what the call allocates is that stream's memory: work still pending on the
    current stream, on memory freed there since, does not reach the results."""
    g = torch.Generator().manual_seed(9)
    hq, hkv, d, bs, n, ctx = 8, 2, 128, 16, 40, 1000
    dt = torch.float16
    nb = -(-(ctx + n) // bs)
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    cache = torch.randn((nb, 2, hkv, bs, d), generator=g).to(dt).cuda()
    q, k, v = (torch.randn((n, h, d), generator=g).to(dt).cuda() for h in (hq, hkv, hkv))
    inv, _ = rope.rope_frequencies(d, device="cuda")
    mask = W.tree_mask([list(range(-1, n - 1))]).cuda()
    pos, cu, before, lens = torch.arange(n, dtype=torch.int32, device="cuda") + ctx, i32([0, n]), i32([ctx]), i32([ctx + n])

    def step(stream):
        turned = pkv.rope_append(cache, q, k, v, inv, cu, before, table, positions=pos, stream=stream)
        return turned, pkv.paged_attn_tree(cache, turned, mask, cu, lens, table, max_q_len=n, stream=stream)

    expect = [t.clone() for t in step(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # two tensors of the results' size and one of the workspace's, freed with writes to them pending
    held = [torch.empty_like(q) for _ in range(2)]
    held.append(torch.empty(pkv.tree_workspace_size(hq, hkv, d, n), dtype=torch.uint8, device="cuda"))
    torch.cuda._sleep(400_000_000)
    for t in held:
        t.fill_(77)
    places = {t.data_ptr() for t in held}
    del held, t
    got = step(side.cuda_stream if as_handle else side)
    assert not places & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(expect, got))
    assert pkv.get_device_error() == 0
