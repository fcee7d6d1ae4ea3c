"""kv_cache_copy and kv_cache_fork, bit for bit, over 16-bit, FP8 and INT8 caches."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref

pytestmark = pytest.mark.gpu
KINDS = ("native", "fp8", "int8")


def pool(kind, nb, heads, bs, d, seed):
    """(cache, scales or None) of random bits."""
    g = torch.Generator().manual_seed(seed)
    shape = (nb, 2, heads, bs, d)
    if kind == "native":
        return torch.randint(-32768, 32768, shape, generator=g, dtype=torch.int16).view(torch.bfloat16), None
    codes = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)
    scales = torch.randn(shape[:3] if kind == "int8" else shape[:4], generator=g)
    return (codes if kind == "int8" else codes.view(torch.float8_e4m3fn)), scales


def bits(t):
    return t.cpu().contiguous().view({2: torch.int16, 1: torch.int8, 4: torch.int32}[t.element_size()]).numpy().copy()


def parts(kind, cache, scales):
    """The arrays of int8_ref.copy_pages."""
    p = [(bits(cache), 3)]
    if kind != "native":
        p.append((bits(scales), 3 if kind == "fp8" else None))
    return p


def same(kind, cache, scales, ref):
    for (x, _), (y, _) in zip(parts(kind, cache, scales), ref):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,bs,d", [(1, 8, 64), (3, 16, 128), (8, 32, 64), (2, 512, 128)])
def test_copy(kind, heads, bs, d):
    nb = 23
    cache, scales = pool(kind, nb, heads, bs, d, bs + d)
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(bs)).to(torch.int32)
    src, dst = order[:9], order[9:18]
    some = torch.tensor([0, bs, 1, bs - 1, bs // 2, 3, 7, 0, bs], dtype=torch.int32)
    for rows in (None, some):
        ref = parts(kind, cache, scales)
        int8_ref.copy_pages(ref, src.tolist(), dst.tolist(), None if rows is None else rows.tolist(), bs)
        c, s = cache.cuda(), None if scales is None else scales.cuda()
        pkv.kv_cache_copy(c, src.cuda(), dst.cuda(), None if rows is None else rows.cuda(), scales=s)
        assert pkv.get_device_error() == 0
        same(kind, c, s, ref)


def test_copy_head_dim_256():
    cache, _ = pool("native", 5, 3, 32, 256, 1)
    c = cache.cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    pkv.kv_cache_copy(c, i(0, 1), i(4, 3), i(17, 32))
    ref = [(bits(cache), 3)]
    int8_ref.copy_pages(ref, [0, 1], [4, 3], [17, 32], 32)
    assert np.array_equal(bits(c), ref[0][0])


@pytest.mark.parametrize("kind", KINDS)
def test_copy_between_pools(kind):
    """One pool's pages into another, of another size; a source page twice."""
    a, sa = pool(kind, 6, 2, 16, 64, 1)
    b, sb = pool(kind, 11, 2, 16, 64, 2)
    src, dst = [5, 0, 5], [10, 3, 0]
    ca, cb = a.cuda(), b.cuda()
    da, db = (None if s is None else s.cuda() for s in (sa, sb))
    pkv.kv_cache_copy(cb, torch.tensor(src, dtype=torch.int32).cuda(), torch.tensor(dst, dtype=torch.int32).cuda(),
                      src_cache=ca, src_scales=da, scales=db)
    assert pkv.get_device_error() == 0
    want, wants = bits(b), None if sb is None else bits(sb)
    want[dst] = bits(a)[src]
    assert np.array_equal(bits(cb), want)
    assert np.array_equal(bits(ca), bits(a))
    if wants is not None:
        wants[dst] = bits(sa)[src]
        assert np.array_equal(bits(db), wants)


def test_copy_skips_what_is_out_of_range():
    cache, scales = pool("int8", 6, 2, 16, 64, 3)
    c, s = cache.cuda(), scales.cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    pkv.kv_cache_copy(c, i(0, 6, -1, 1, 2), i(3, 4, 5, -1, 6), scales=s)
    assert pkv.get_device_error() == 5
    want = bits(cache)
    want[3] = want[0]
    assert np.array_equal(bits(c), want)
    pkv.kv_cache_copy(c, i(1, 2), i(4, 5), i(17, -1), scales=s)
    assert pkv.get_device_error() == 5
    assert np.array_equal(bits(c), want)
    pkv.kv_cache_copy(c, i(), i(), scales=s)
    assert pkv.get_device_error() == 0


def test_copy_offsets_beyond_32_bits():
    nb = 5000
    c = torch.zeros((nb, 2, 32, 128, 128), dtype=torch.int8, device="cuda")   # 5.2 GB
    s = torch.zeros((nb, 2, 32), device="cuda")
    c[0] = torch.arange(128, device="cuda", dtype=torch.int8)
    c[nb - 2], s[nb - 2], s[0] = 5, 2.0, 1.0
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    pkv.kv_cache_copy(c, i(0, nb - 2), i(nb - 1, 1), scales=s)
    assert pkv.get_device_error() == 0
    assert torch.equal(c[nb - 1], c[0]) and torch.equal(c[1], c[nb - 2])
    assert s[nb - 1].eq(1).all() and s[1].eq(2).all() and not c[2:nb - 2].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,bs,d", [(1, 8, 64), (3, 16, 128), (2, 512, 64)])
def test_fork(kind, heads, bs, d):
    """Empty, one-token, full and partly filled parents, several children and none, children that go on in place."""
    lens = [0, 1, bs, 2 * bs + 3, 3 * bs - 1, 4 * bs]
    mb, nb = 4, 40
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(d)).tolist()
    tables = torch.full((len(lens), mb), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for j in range(-(-n // bs)):
            tables[b, j] = order.pop()
    parents = torch.tensor([3, 3, 0, 1, 4, 4, 5, 2, 2, 3], dtype=torch.int32)
    fresh = torch.tensor([order.pop() for _ in parents], dtype=torch.int32)
    fresh[4], fresh[8] = -1, -1
    cache, scales = pool(kind, nb, heads, bs, d, 7)
    ref = parts(kind, cache, scales)
    want, want_lens = int8_ref.fork(ref, tables.numpy(), lens, parents.tolist(), fresh.tolist(), bs)
    c, s = cache.cuda(), None if scales is None else scales.cuda()
    out, out_lens = pkv.kv_cache_fork(c, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), parents.cuda(),
                                      fresh.cuda(), scales=s)
    assert pkv.get_device_error() == 0
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(out_lens.cpu().numpy(), want_lens)
    same(kind, c, s, ref)


def test_fork_long_tables():
    """Tables of several thousand pages, their rows written by several blocks."""
    mb, bs, n, m = 5000, 8, 3, 40
    nb = n * mb + m
    c = torch.randint(-100, 100, (nb, 2, 1, bs, 64), dtype=torch.int8).cuda()
    s = torch.ones((nb, 2, 1), device="cuda")
    before = c.clone()
    tables = torch.arange(n * mb, dtype=torch.int32).reshape(n, mb)
    lens = torch.tensor([mb * bs, 1025 * bs + 3, 4999 * bs + 7], dtype=torch.int32)
    parents = torch.arange(m, dtype=torch.int32) % n
    fresh = torch.arange(n * mb, nb, dtype=torch.int32)
    out, out_lens = pkv.kv_cache_fork(c, tables.cuda(), lens.cuda(), parents.cuda(), fresh.cuda(), scales=s)
    assert pkv.get_device_error() == 0
    ref = [(before.cpu().numpy().copy(), 3)]
    want, want_lens = int8_ref.fork(ref, tables.numpy(), lens.tolist(), parents.tolist(), fresh.tolist(), bs)
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(out_lens.cpu().numpy(), want_lens)
    assert np.array_equal(c.cpu().numpy(), ref[0][0])


def test_fork_flags_what_is_out_of_range():
    cache, scales = pool("int8", 8, 2, 16, 64, 5)
    c, s = cache.cuda(), scales.cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    tables = i([0, 1], [2, 77], [3, 4])
    lens = i(33, 20, 20)
    # a parent with a length beyond its table; parents that do not exist; a last page outside the pool; a new page outside
    for parent, new, want, n in ((0, 5, [-1, -1], 0), (-1, 5, [-1, -1], 0), (3, 5, [-1, -1], 0), (1, 5, [2, 5], 20),
                                 (2, 8, [3, -1], 20)):
        out, out_lens = pkv.kv_cache_fork(c, tables, lens, i(parent), i(new), scales=s)
        assert pkv.get_device_error() == 5
        assert out.tolist() == [want] and out_lens.tolist() == [n]
    assert np.array_equal(bits(c), bits(cache)) and np.array_equal(bits(s), bits(scales))
    # the others of the call are served
    out, out_lens = pkv.kv_cache_fork(c, tables, lens, i(0, 2), i(5, 6), scales=s)
    assert pkv.get_device_error() == 5
    assert out.tolist() == [[-1, -1], [3, 6]] and out_lens.tolist() == [0, 20]
    assert np.array_equal(bits(c)[6, :, :, :4], bits(cache)[4, :, :, :4]) and torch.equal(s[6].cpu(), scales[4])
    assert np.array_equal(bits(c)[6, :, :, 4:], bits(cache)[6, :, :, 4:])


def test_binding_refuses():
    cache, scales = pool("int8", 4, 2, 16, 64, 1)
    c, s = cache.cuda(), scales.cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    for bad in (dict(src_pages=i(0, 1)), dict(src_pages=i(0).long()), dict(src_pages=i(0).cpu()), dict(num_rows=i(1, 2)),
                dict(scales=None), dict(src_scales=s), dict(src_cache=c[:, :, :1].contiguous(), src_scales=s),
                dict(src_cache=c), dict(src_cache=c.view(torch.uint8), src_scales=s)):
        with pytest.raises((ValueError, TypeError)):
            pkv.kv_cache_copy(c, **{**dict(src_pages=i(0), dst_pages=i(1), scales=s), **bad})
    t = i([0, 1])
    for bad in (dict(context_lens=i(3, 4)), dict(new_pages=i(2, 3)), dict(parents=i(0).long()), dict(out_tables=i([0])),
                dict(out_lens=i(0, 0)), dict(scales=None)):
        with pytest.raises((ValueError, TypeError)):
            pkv.kv_cache_fork(c, **{**dict(block_tables=t, context_lens=i(3), parents=i(0), new_pages=i(2), scales=s), **bad})
    with pytest.raises(pkv.PkvError):
        pkv.kv_cache_fork(c, t, i(3), i(0), i(2), out_tables=t, scales=s)
