"""paged_attn_decode over an INT8 cache against the plain implementation in 64 bits.

The bounds follow from the arithmetic (see `bounds`): products of f16 query elements and integer codes are exact in FP32 and
summed there; the weights enter the product with V as two f16 parts; the output is rounded once."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def pool(nb, heads, bs, d, seed, spread=2):
    """Codes of normal values, scales around 2^-5 that differ between pages by 2^-spread to 2^spread."""
    g = torch.Generator().manual_seed(seed)
    codes = (torch.randn((nb, 2, heads, bs, d), generator=g) * 36).round().clamp(-127, 127).to(torch.int8)
    e = torch.randint(-spread, spread + 1, (nb, 2, heads), generator=g) - 5
    return codes, torch.ldexp(torch.ones((nb, 2, heads)), e)


def tables_of(lens, bs, nb, mb, seed):
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(seed)).tolist()
    t = torch.full((len(lens), mb), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // bs)):
            t[b, i] = order.pop()
    return t


def bounds(codes, scales, q, cu, lens, tables, scale, out, weight_eps, causal=True, weight_abs=2.0 ** -36):
    """Elementwise bounds (out, lse) of an FP32 result before its rounding.

    Scores: D exact products summed in FP32 (the tensor core's sums truncate: 2^-23 a step) and scaled: their error is
    at most e = (D + 4) 2^-23 scale sum |q||k|, and an element of q below f16's normal range is off by 2^-25, so
    e += D 2^-25 scale max|k|. A weight is then off by a factor within 2 e + 2^-20 (ex2: 2^-22, running maxima and
    the sums 2^-23 a step over the tiles of a warp: L / 128 steps, and the split's merge) + weight_eps (its rounding),
    so the output by that times sum p |v| / sum p, and as much again for the sum it is divided by.

    f16 has no step below 2^-24, so a weight that goes into the product 2^k times itself (k = 11 in the decode, 7 in the
    prefill), relative to a past maximum that is never above the row's, is off by 2^-25 2^-k = weight_abs of the row's largest
    weight besides: over n keys of at most 127 steps of the context's largest V scale, by n weight_abs 127 max sv, over
    sum p >= 1."""
    heads, d = codes.shape[2], codes.shape[4]
    group = q.shape[1] // heads
    err, err_lse = np.zeros(out.shape), np.zeros(out.shape[:2])
    for b, length in enumerate(lens):
        length, r0, n = int(length), int(cu[b]), int(cu[b + 1] - cu[b])
        if length == 0 or n == 0:
            continue
        kv = int8_ref.context(codes, scales, tables[b], length)
        for h in range(q.shape[1]):
            k, v = kv[0, h // group], kv[1, h // group]
            x = q[r0:r0 + n, h]
            s = x @ k.T * scale
            if causal:
                for r in range(n):
                    s[r, length - n + r + 1:] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            e = ((d + 4) * 2.0 ** -23 * (np.abs(x) @ np.abs(k).T).max(1) + d * 2.0 ** -25 * np.abs(k).max()) * abs(scale)
            eps = 2 * e + 2.0 ** -20 + length / 128 * 2.0 ** -23 + weight_eps
            pages = [int(i) for i in tables[b][:-(-length // codes.shape[3])]]
            below = length * weight_abs * 127 * float(scales[pages, 1, h // group].max())
            err[r0:r0 + n, h] = (2 * eps[:, None] * (p @ np.abs(v)) + below) / p.sum(1, keepdims=True)
            err_lse[r0:r0 + n, h] = eps + 2.0 ** -22 * (1 + np.abs(s.max(1)))
    return err, err_lse


def check(out, lse, ref, ref_lse, err, err_lse):
    """out (of any type) within err and half a step of its type; lse within err_lse."""
    half = torch.finfo(out.dtype).eps / 2
    got = out.double().cpu().numpy()
    tiny = torch.finfo(out.dtype).smallest_normal * half * 2
    assert np.all(np.isfinite(got))
    worst = np.abs(got - ref) - (err + half * (np.abs(ref) + err) + tiny)
    assert worst.max(initial=-1) <= 0, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
    if lse is not None:
        got = lse.double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(ref_lse))
        seen = ~np.isneginf(ref_lse)
        assert np.all(np.abs(got[seen] - ref_lse[seen]) <= err_lse[seen])


def run(lens, hq, heads, d, bs, dtype, seed, out_dtype=None, num_splits=0, spread=2, scale=None, codes=None, scales=None):
    mb = max(1, max(-(-n // bs) for n in lens)) + 1
    nb = sum(-(-n // bs) for n in lens) + 2
    if codes is None:
        codes, scales = pool(nb, heads, bs, d, seed, spread)
    tables = tables_of(lens, bs, codes.shape[0], mb, seed)
    q = torch.randn((len(lens), hq, d), generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    scale = d ** -0.5 if scale is None else scale
    lse = torch.empty((len(lens), hq), device="cuda")
    out = pkv.paged_attn_decode(codes.cuda(), q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale=scale,
                                num_splits=num_splits, out_dtype=None if out_dtype is None else torch.float32, lse=lse,
                                scales=scales.cuda())
    assert pkv.get_device_error() == 0
    cu = np.arange(len(lens) + 1)
    args = (codes.numpy(), scales.numpy(), q.double().numpy(), cu, lens, tables.numpy(), scale)
    ref, ref_lse = int8_ref.attention(*args, causal=False)
    # more than 8 heads per KV head: the weights may be rounded once to f16 (half a step, 2^-11), times 2^7
    wide = hq // heads > 8
    err, err_lse = bounds(*args, ref, 2.0 ** -11 if wide else 2.0 ** -21, causal=False,
                          weight_abs=2.0 ** -32 if wide else 2.0 ** -36)
    check(out, lse, ref, ref_lse, err, err_lse)


@pytest.mark.parametrize("num_splits", [0, 1, 9])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128, 512])
def test_lengths(bs, d, num_splits):
    """Empty and one-token contexts, ones that end inside a page, a tile, a warp's share, a split or a CTA's run."""
    run([0, 1, bs - 1, bs, bs + 1, 31, 32, 33, 127, 129, 700, 1537], 4, 2, d, bs, "bf16", bs + d, num_splits=num_splits)


@pytest.mark.parametrize("lens", [[5000], [1], [0], [17, 3000], [900, 0, 0, 33], [100] * 9, [2000] * 20, [600] * 40, [40] * 200])
@pytest.mark.parametrize("hq,heads", [(4, 1), (8, 8), (7, 1), (16, 1), (40, 1)])
def test_batches(lens, hq, heads):
    """From one sequence to many: clusters of every size, and the splits."""
    run(lens, hq, heads, 128, 16, "f16", len(lens) + hq)


@pytest.mark.parametrize("hq,heads", [(1, 1), (4, 2), (6, 2), (4, 1), (10, 2), (6, 1), (21, 3), (8, 1), (9, 1), (13, 1), (32, 2),
                                      (24, 2), (34, 2), (32, 32)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("num_splits", [0, 3])
def test_groups(hq, heads, d, num_splits):
    run([300, 0, 45, 1000], hq, heads, d, 16, "f16", hq + d, num_splits=num_splits)


@pytest.mark.parametrize("num_splits", [1, 2, 5, 40])
@pytest.mark.parametrize("hq", [8, 24])
def test_splits(num_splits, hq):
    run([3000, 17, 1, 0, 129], hq, 2, 128, 32, "bf16", num_splits, num_splits=num_splits)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("hq", [12, 33, 128, 130])
def test_many_heads(bs, d, hq):
    """One KV head for many query heads: lengths around tiles, one tile, an odd and an even number of them."""
    run([0, 1, bs, 127, 128, 129, 256, 257, 400, 1000, 1537], hq, 1, d, bs, "bf16" if bs == 16 else "f16", bs + hq, num_splits=2)


def test_many_heads_float32_and_scales():
    run([300, 900], 16, 1, 128, 16, "f16", 5, out_dtype=torch.float32, num_splits=1)
    run([500, 64, 900], 20, 1, 128, 16, "bf16", 8, spread=6, scale=0.01, num_splits=1)
    codes, scales = pool(60, 2, 8, 64, 9)
    scales[::3, 1] = 0.0
    run([200, 150], 24, 2, 64, 8, "bf16", 9, codes=codes, scales=scales, num_splits=1)
    run([200, 150], 24, 2, 64, 8, "bf16", 9, codes=codes, scales=torch.zeros_like(scales), num_splits=1)
    run([200, 150], 24, 2, 64, 8, "bf16", 9, scale=-0.2, num_splits=1)
    run([200, 150], 24, 2, 64, 8, "bf16", 9, scale=0.0, num_splits=1)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_float32_output(dtype):
    run([1000, 40, 3], 8, 2, 128, 16, dtype, 3, out_dtype=torch.float32)


def test_page_scales_far_apart():
    """Pages whose scales differ by 2^20, V's zero among them; scales that are no powers of two."""
    run([500, 64, 900], 4, 2, 128, 16, "f16", 8, spread=10, scale=0.002)
    codes, scales = pool(60, 2, 8, 64, 9)
    scales[::3, 1] = 0.0
    run([200, 150], 4, 2, 64, 8, "bf16", 9, codes=codes, scales=scales)
    scales = torch.rand((60, 2, 2), generator=torch.Generator().manual_seed(4)) * 0.05 + 0.001
    run([200, 150], 4, 2, 64, 8, "bf16", 9, codes=codes, scales=scales)


def test_small_weights_add_up():
    """One key far above 30000 others, each of whose weights alone is below f16's range: together they count."""
    d, bs, n = 64, 64, 30016
    codes = torch.zeros((n // bs, 2, 1, bs, d), dtype=torch.int8)
    codes[:, 1] = 100
    codes[0, 0, 0, 0], codes[0, 1, 0, 0] = 64, -100
    scales = torch.ones((n // bs, 2, 1)) / 64
    tables = torch.arange(n // bs, dtype=torch.int32)[None]
    q = torch.full((1, 1, d), 18.0 / d)                        # the first key's score is 18, the others' 0
    out = pkv.paged_attn_decode(codes.cuda(), q.half().cuda(), tables.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                                scale=1.0, out_dtype=torch.float32, scales=scales.cuda())
    rest = (n - 1) * math.exp(-18.0 * float(torch.tensor(18.0 / d).half()) * d / 18.0)
    want = 100 / 64 * (rest - 1) / (rest + 1)
    assert abs(out[0, 0, 0].item() - want) <= 2e-5, (out[0, 0, 0].item(), want)


def test_what_is_not_a_number():
    """A NaN scale reaches the sequences that see its page, and no other; what lies behind a context's end reaches none."""
    codes, scales = pool(8, 1, 128, 64, 3)
    tables = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32)
    scales[0, 0], scales[3, 1] = float("nan"), float("nan")
    scales[5], codes[4, :, :, 60:] = float("nan"), 127
    lens = torch.tensor([256, 256, 60, 200], dtype=torch.int32)
    for splits, heads in ((0, 2), (1, 2), (2, 2), (1, 20), (2, 20)):
        q = torch.randn((4, heads, 64), generator=torch.Generator().manual_seed(1)).half()
        lse = torch.empty((4, heads), device="cuda")
        out = pkv.paged_attn_decode(codes.cuda(), q.cuda(), tables.cuda(), lens.cuda(), lse=lse, num_splits=splits,
                                    scales=scales.cuda())
        assert torch.isnan(out[:2]).all() and torch.isfinite(out[2:]).all()
        assert torch.isnan(lse[0]).all() and torch.isfinite(lse[2:]).all()
    ref, _ = int8_ref.attention(codes.numpy(), np.nan_to_num(scales.numpy()), q.double().numpy(), range(5), lens.tolist(),
                                tables.numpy(), 0.125, causal=False)
    assert np.abs(out[2:].double().cpu().numpy() - ref[2:]).max() < 1e-2


def test_bad_pages_are_flagged():
    codes, scales = pool(4, 1, 16, 64, 3)
    q = torch.randn((2, 1, 64)).half().cuda()
    tables = torch.tensor([[0, 7], [2, 1]], dtype=torch.int32).cuda()
    out = pkv.paged_attn_decode(codes.cuda(), q, tables, torch.tensor([20, 20], dtype=torch.int32).cuda(), scales=scales.cuda())
    assert pkv.get_device_error() == 5
    assert torch.isfinite(out[1]).all()


def test_step_is_decode_then_append():
    lens = [33, 0, 700, 15, 16]
    codes, scales = pool(70, 2, 16, 128, 5)
    tables = tables_of([n + 1 for n in lens], 16, 70, 46, 5).cuda()
    ctx = torch.tensor(lens, dtype=torch.int32).cuda()
    q, k, v = (torch.randn((5, h, 128), generator=torch.Generator().manual_seed(h)).bfloat16().cuda() for h in (8, 2, 2))
    v = v * 3
    c1, s1, c2, s2 = codes.cuda(), scales.cuda(), codes.cuda(), scales.cuda()
    out1 = pkv.paged_attn_decode_step(c1, q, tables, ctx, k, v, scales=s1)
    out2 = pkv.paged_attn_decode(c2, q, tables, ctx, scales=s2)
    pkv.kv_cache_append(c2, k, v, torch.arange(6, dtype=torch.int32).cuda(), ctx, tables, scales=s2)
    assert pkv.get_device_error() == 0
    assert torch.equal(out1, out2) and torch.equal(c1, c2) and torch.equal(s1, s2)
    out3 = pkv.paged_attn_decode_noalloc(codes.cuda(), q, tables, ctx, scales=scales.cuda())
    assert torch.equal(out1, out3)


def test_large_batch_and_shared_pages():
    """More sequences than a launch's tables hold; every sequence reads the same pages."""
    n = 2500
    codes, scales = pool(6, 1, 8, 64, 5)
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 41, (n,), generator=g, dtype=torch.int32)
    tables = torch.stack([torch.randperm(6, generator=g)[:5] for _ in range(n)]).to(torch.int32)
    q = torch.randn((n, 1, 64), generator=g).half()
    lse = torch.empty((n, 1), device="cuda")
    out = pkv.paged_attn_decode(codes.cuda(), q.cuda(), tables.cuda(), lens.cuda(), lse=lse, scales=scales.cuda())
    args = (codes.numpy(), scales.numpy(), q.double().numpy(), np.arange(n + 1), lens.tolist(), tables.numpy(), 0.125)
    ref, ref_lse = int8_ref.attention(*args, causal=False)
    check(out, lse, ref, ref_lse, *bounds(*args, ref, 2.0 ** -21, causal=False))


def test_offsets_beyond_32_bits():
    nb, heads = 2600, 64
    codes = torch.zeros((nb, 2, heads, 128, 128), dtype=torch.int8, device="cuda")
    scales = torch.zeros((nb, 2, heads), device="cuda")
    c, s = pool(2, heads, 128, 128, 6)
    codes[-2:], scales[-2:] = c.cuda(), s.cuda()
    q = torch.randn((1, heads, 128), generator=torch.Generator().manual_seed(1)).half()
    out = pkv.paged_attn_decode(codes, q.cuda(), torch.tensor([[nb - 1, nb - 2]], dtype=torch.int32).cuda(),
                                torch.tensor([200], dtype=torch.int32).cuda(), scales=scales)
    args = (c.numpy(), s.numpy(), q.double().numpy(), [0, 1], [200], np.array([[1, 0]]), 128 ** -0.5)
    ref, ref_lse = int8_ref.attention(*args, causal=False)
    check(out, None, ref, ref_lse, *bounds(*args, ref, 2.0 ** -21, causal=False))


def test_in_a_graph():
    codes, scales = pool(40, 2, 16, 128, 5)
    tables = tables_of([300, 200], 16, 40, 20, 5).cuda()
    lens = torch.tensor([300, 200], dtype=torch.int32).cuda()
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(1)).half().cuda()
    c, s = codes.cuda(), scales.cuda()
    want = pkv.paged_attn_decode(c, q, tables, lens, scales=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkv.paged_attn_decode(c, q, tables, lens, scales=s)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_binding_refuses():
    codes, scales = (x.cuda() for x in pool(4, 2, 16, 64, 1))
    q = torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda")
    t, n = torch.zeros((1, 2), dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    for bad in (dict(q=q[..., :32].contiguous()), dict(context_lens=n.repeat(2)), dict(block_tables=t.cpu()), dict(scales=None),
                dict(scales=scales[:2].contiguous()), dict(lse=torch.empty((1, 3), device="cuda")),
                dict(lse=torch.empty((1, 4), dtype=torch.float16, device="cuda")), dict(out=torch.empty((1, 4, 32), device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            pkv.paged_attn_decode(codes, **{**dict(q=q, block_tables=t, context_lens=n, scales=scales), **bad})
    with pytest.raises(pkv.PkvError):
        pkv.paged_attn_decode(codes, q[:, :3].contiguous(), t, n, scales=scales)
