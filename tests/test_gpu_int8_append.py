"""kv_cache_append into an INT8 cache, bit for bit against the plain implementation in 64 bits: codes, scales, every row
that the call has no business with."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def pool(nb, heads, bs, d, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-127, 128, (nb, 2, heads, bs, d), generator=g, dtype=torch.int8)
    scales = torch.ldexp(torch.ones((nb, 2, heads)), torch.randint(-8, -3, (nb, 2, heads), generator=g))
    return codes, scales


def tables_of(lens, bs, nb, mb, seed):
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).tolist()
    t = torch.full((len(lens), mb), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // bs)):
            t[b, i] = order.pop()
    return t


def run(codes, scales, k, v, cu, ctx, tables, expect_error=0):
    """The call on copies of the pool against the reference on others; returns the GPU's codes and scales."""
    dc, ds = codes.cuda(), scales.cuda()
    pkv.kv_cache_append(dc, k.cuda(), v.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                        torch.tensor(ctx, dtype=torch.int32).cuda(), tables.cuda(), scales=ds)
    assert pkv.get_device_error() == expect_error
    rc, rs = codes.numpy().copy(), scales.numpy().copy()
    int8_ref.append(rc, rs, k.double().numpy(), v.double().numpy(), cu, ctx, tables.numpy())
    gc, gs = dc.cpu().numpy(), ds.cpu().numpy()
    assert np.array_equal(gs, rs, equal_nan=True), np.argwhere(gs != rs)[:8]
    assert np.array_equal(gc, rc), np.argwhere(gc != rc)[:8]
    return dc.cpu(), ds.cpu()


def rows(total, heads, d, dtype, seed, spread=3.0):
    """Rows of magnitudes that differ by factors, so that scales grow, stay and start low."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((2, total, heads, d), generator=g)
    x *= torch.exp2(torch.randn((2, total, heads, 1), generator=g) * spread)
    return x.to(DT[dtype]).unbind(0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128, 256, 512])
def test_ragged_prompts(bs, d):
    """Fresh sequences, half-filled first pages, pages that end inside, empty and one-token sequences; pages by the
    prompt's length and by the token."""
    for seed, new, ctx in ((1, [700, 0, 1, 33, 2 * bs, bs - 1], [0, 5, 3 * bs - 1, bs // 2, bs, 2 * bs + 1]),
                           (2, [1, 1, 0, 2, 1], [0, bs - 1, 4, bs - 1, bs]),
                           (3, [bs], [0])):
        heads, dtype = 3, ("f16", "bf16")[seed % 2]
        lens = [n + c for n, c in zip(new, ctx)]
        mb = max(-(-n // bs) for n in lens) + 1
        nb = sum(-(-n // bs) for n in lens) + 2
        codes, scales = pool(nb, heads, bs, d, seed)
        k, v = rows(sum(new), heads, d, dtype, seed)
        run(codes, scales, k, v, np.concatenate(([0], np.cumsum(new))).tolist(), ctx,
            tables_of(lens, bs, nb, mb, seed))


@pytest.mark.parametrize("batch", [33, 100, 1500])
def test_many_sequences(batch):
    g = np.random.default_rng(batch)
    new, ctx = g.integers(0, 4, batch).tolist(), g.integers(0, 50, batch).tolist()
    lens = [n + c for n, c in zip(new, ctx)]
    nb = sum(-(-n // 16) for n in lens) + 1
    codes, scales = pool(nb, 1, 16, 64, batch)
    k, v = rows(sum(new), 1, 64, "bf16", batch)
    run(codes, scales, k, v, np.concatenate(([0], np.cumsum(new))).tolist(), ctx, tables_of(lens, 16, nb, 6, batch))


def test_one_token_after_another():
    """64 decode steps: the pool after each is the reference's."""
    codes, scales = pool(10, 2, 16, 128, 7)
    tables = tables_of([80, 64], 16, 10, 5, 7)
    for t in range(64):
        k, v = rows(2, 2, 128, "f16", 100 + t, spread=1.0)
        codes, scales = run(codes, scales, k, v, [0, 1, 2], [t + 3, t], tables)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_ends_of_the_range(dtype):
    """Zeros, the smallest and the largest values, magnitudes at the border between two scales, ties."""
    d, bs = 64, 16
    t = DT[dtype]
    k, v = (torch.zeros((64, 1, d), dtype=t) for _ in range(2))
    info = torch.finfo(t)
    k[16:32] = info.smallest_normal * 2.0 ** (-6 if dtype == "bf16" else -9)   # subnormal
    k[32, 0, 0], k[33, 0, 5] = info.max, -info.max
    v[0:16, 0] = torch.arange(-32, 32).to(t) / 2 + 0.25
    v[15, 0, 0] = 127.0                                                       # scale 1: ties at .5 and quarters
    v[16, 0, 0] = 127.5 if dtype == "f16" else 128.0                          # scale 2
    v[17, 0] = torch.arange(64).to(t)
    v[32:48] = info.tiny
    codes, scales = pool(6, 1, bs, d, 3)
    run(codes, scales, k, v, [0, 64], [0], torch.tensor([[4, 2, 0, 1]], dtype=torch.int32))
    # behind older rows whose scale is 0, tiny, huge or not a power of two
    for old in (0.0, 2.0 ** -126, 2.0 ** 122, 0.0371):
        codes, scales = pool(2, 1, bs, d, 4)
        scales[1] = old
        run(codes, scales, k[15:18].contiguous(), v[15:18].contiguous(), [0, 3], [9], torch.tensor([[1]], dtype=torch.int32))


@pytest.mark.parametrize("old", [1e-45, 1e-40, 2.0 ** -127])
def test_an_older_scale_below_the_range(old):
    """It counts as 0: rows of zeros leave 0, others start the page's scale, older codes become 0."""
    codes, scales = pool(3, 1, 16, 64, 4)
    scales[1:] = old
    k, v = torch.zeros((2, 3, 1, 64), dtype=torch.bfloat16)
    k[1, 0, 3], v[2, 0, 5] = 1e-38, -2e-39
    run(codes, scales, k, v, [0, 3], [9], torch.tensor([[1]], dtype=torch.int32))
    run(codes, scales, v * 0, k * 0, [0, 3], [9], torch.tensor([[2]], dtype=torch.int32))


def test_what_is_not_a_number():
    """A NaN or an infinity makes its page's scale NaN, stays so, and leaves with the page's next start."""
    codes, scales = pool(4, 2, 16, 64, 9)
    tables = torch.tensor([[3, 1]], dtype=torch.int32)
    k, v = rows(20, 2, 64, "bf16", 9)
    k[4, 0, 63], v[18, 1, 0] = float("nan"), float("-inf")
    codes, scales = run(codes, scales, k, v, [0, 20], [0], tables)
    assert torch.isnan(scales[3, 0, 0]) and torch.isnan(scales[1, 1, 1]) and int(torch.isnan(scales).sum()) == 2
    k, v = rows(4, 2, 64, "bf16", 10)
    codes, scales = run(codes, scales, k, v, [0, 4], [20], tables)
    assert torch.isnan(scales[1, 1, 1])
    codes, scales = run(codes, scales, k, v, [0, 4], [16], tables)
    assert not torch.isnan(scales[1]).any()


def test_bad_pages_and_padding_rows():
    """Positions without a page of the pool are flagged and skipped; rows at or behind cu_new_lens[batch] are nobody's."""
    codes, scales = pool(4, 2, 16, 128, 11)
    k, v = rows(70, 2, 128, "f16", 11)
    # sequence 0: a page outside the pool in the middle; sequence 1: behind its table
    tables = torch.tensor([[0, 99, 2], [3, -1, -1]], dtype=torch.int32)
    run(codes, scales, k, v, [0, 40, 45], [0, 46], tables, expect_error=5)
    run(codes, scales, k, v, [0, 0, 0], [0, 3], tables)
    run(codes, scales, k, v, [0, 1, 5], [3, 6], tables)


def test_offsets_beyond_32_bits():
    """A pool of 5 GB: its last pages."""
    nb, heads, bs, d = 2600, 64, 128, 128
    cache = torch.zeros((nb, 2, heads, bs, d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((nb, 2, heads), device="cuda")
    k, v = rows(130, heads, d, "bf16", 13)
    tables = torch.tensor([[nb - 1, nb - 2]], dtype=torch.int32)
    pkv.kv_cache_append(cache, k.cuda(), v.cuda(), torch.tensor([0, 130], dtype=torch.int32).cuda(),
                        torch.tensor([5], dtype=torch.int32).cuda(), tables.cuda(), scales=scales)
    assert pkv.get_device_error() == 0
    rc, rs = np.zeros((2, 2, heads, bs, d), np.int8), np.zeros((2, 2, heads), np.float32)
    int8_ref.append(rc, rs, k.double().numpy(), v.double().numpy(), [0, 130], [5], np.array([[1, 0]], np.int32))
    assert np.array_equal(cache[-2:].cpu().numpy(), rc) and np.array_equal(scales[-2:].cpu().numpy(), rs)
    assert not cache[:-2].any()


def test_in_a_graph_and_on_a_stream():
    codes, scales = pool(6, 2, 32, 128, 15)
    tables = torch.tensor([[4, 0], [1, 5]], dtype=torch.int32)
    args = [torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 40, 41], [3, 31])]
    k, v = (x.cuda() for x in rows(41, 2, 128, "bf16", 15))
    dc, ds, t = codes.cuda(), scales.cuda(), tables.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.kv_cache_append(dc, k, v, args[0], args[1], t, scales=ds, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_cache_append(dc, k, v, args[0], args[1], t, scales=ds)
    for seed in (16, 17):
        k2, v2 = rows(41, 2, 128, "bf16", seed)
        k.copy_(k2.cuda()), v.copy_(v2.cuda()), dc.copy_(codes.cuda()), ds.copy_(scales.cuda())
        graph.replay()
        rc, rs = codes.numpy().copy(), scales.numpy().copy()
        int8_ref.append(rc, rs, k2.double().numpy(), v2.double().numpy(), [0, 40, 41], [3, 31], tables.numpy())
        assert np.array_equal(dc.cpu().numpy(), rc) and np.array_equal(ds.cpu().numpy(), rs)


def test_binding_refuses():
    codes, scales = (x.cuda() for x in pool(4, 2, 16, 64, 1))
    k, v = (x.cuda() for x in rows(3, 2, 64, "f16", 1))
    cu, ctx, t = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 3], [0], [[0]]))
    call = lambda **kw: pkv.kv_cache_append(codes, **{**dict(k_new=k, v_new=v, cu_new_lens=cu, ctx_before=ctx, block_tables=t,
                                                             scales=scales), **kw})
    with pytest.raises(ValueError):
        call(k_new=k[:, :1].contiguous(), v_new=v[:, :1].contiguous())
    with pytest.raises(ValueError):
        call(cu_new_lens=cu[:1])
    with pytest.raises(ValueError):
        call(ctx_before=ctx.cpu())
    with pytest.raises(ValueError):
        call(k_new=k.cpu(), v_new=v.cpu())
    with pytest.raises(ValueError):
        call(scales=scales[:, :, :1].contiguous())
    with pytest.raises(pkv.PkvError):
        call(k_new=k.float(), v_new=v.float())
