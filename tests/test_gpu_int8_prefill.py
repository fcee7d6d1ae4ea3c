"""paged_attn_prefill and paged_attn_mixed over an INT8 cache against the plain implementation in 64 bits. Bounds: those of
the decode (tests/test_gpu_int8_decode.py) with the weights rounded once to f16 (half a step, 2^-11)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref
from tests.test_gpu_int8_decode import DT, bounds, check, pool, tables_of

pytestmark = pytest.mark.gpu


def run(lens, new, hq, heads, d, bs, dtype, seed, causal=True, out_dtype=None, spread=2, scale=None, codes=None, scales=None,
        mixed=False):
    mb = max(1, max(-(-n // bs) for n in lens)) + 1
    nb = sum(-(-n // bs) for n in lens) + 2
    if codes is None:
        codes, scales = pool(nb, heads, bs, d, seed, spread)
    tables = tables_of(lens, bs, codes.shape[0], mb, seed)
    cu = np.concatenate(([0], np.cumsum(new)))
    pad = 3                                                    # rows behind the last sequence: left as they were
    q = torch.randn((int(cu[-1]) + pad, hq, d), generator=torch.Generator().manual_seed(seed + 1)).to(DT[dtype])
    scale = d ** -0.5 if scale is None else scale
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=out_dtype or DT[dtype], device="cuda")
    dev = [torch.tensor(np.asarray(x), dtype=torch.int32).cuda() for x in (cu, lens)]
    fn = pkv.paged_attn_mixed if mixed else pkv.paged_attn_prefill
    fn(codes.cuda(), q.cuda(), dev[0], dev[1], tables.cuda(), max_q_len=max(new), scale=scale, causal=causal, out=out, lse=lse,
       scales=scales.cuda())
    assert pkv.get_device_error() == 0
    assert out[cu[-1]:].eq(7).all() and lse[cu[-1]:].eq(7).all()
    args = (codes.numpy(), scales.numpy(), q[:cu[-1]].double().numpy(), cu, lens, tables.numpy(), scale)
    ref, ref_lse = int8_ref.attention(*args, causal=causal)
    err, err_lse = bounds(*args, ref, 2.0 ** -11, causal=causal, weight_abs=2.0 ** -32)
    check(out[:cu[-1]], lse[:cu[-1]], ref, ref_lse, err, err_lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 64, 128, 512])
def test_lengths(bs, d):
    """Chunks of one row, of whole prompts, that end inside a page, a row tile, a key tile; behind contexts of any length."""
    run([1, 40, 129, 300, 257, 700], [1, 7, 129, 1, 256, 300], 4, 2, d, bs, "bf16", bs + d)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_causal_or_not(causal, dtype):
    run([500, 130], [200, 130], 4, 2, 128, 32, dtype, 3, causal=causal)


@pytest.mark.parametrize("hq,heads", [(1, 1), (6, 2), (5, 1), (16, 1), (3, 3)])
def test_groups(hq, heads):
    run([300, 45], [128, 45], hq, heads, 64, 16, "f16", hq)


def test_long_context():
    run([5000], [300], 4, 2, 128, 16, "bf16", 4)


def test_float32_output():
    run([600, 40], [300, 40], 4, 2, 128, 16, "bf16", 5, out_dtype=torch.float32)


def test_page_scales_far_apart():
    """Powers of two that differ by 2^12, V's zero among them; scales that are no powers of two; all scales 0."""
    run([500, 64], [100, 64], 4, 2, 128, 16, "f16", 8, spread=6, scale=0.01)
    codes, scales = pool(60, 2, 8, 64, 9)
    scales[::3, 1] = 0.0
    run([200, 150], [70, 150], 4, 2, 64, 8, "bf16", 9, codes=codes, scales=scales)
    run([200, 150], [70, 150], 4, 2, 64, 8, "bf16", 9, codes=codes, scales=torch.zeros_like(scales))


def test_scales_that_are_no_powers_of_two():
    """Keys and values are then f16 roundings of code times scale: 2 x 2^-11 and 2^-25 of the largest, on both sides."""
    codes, _ = pool(60, 2, 16, 128, 9)
    scales = torch.rand((60, 2, 2), generator=torch.Generator().manual_seed(4)) * 0.05 + 0.001
    lens, new = [200, 350], [70, 350]
    tables = tables_of(lens, 16, 60, 23, 1)
    cu = np.array([0, 70, 420])
    q = torch.randn((420, 4, 128), generator=torch.Generator().manual_seed(5)).half()
    out = pkv.paged_attn_prefill(codes.cuda(), q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), tables.cuda(), max_q_len=350, scales=scales.cuda(),
                                 out_dtype=torch.float32)
    args = (codes.numpy(), scales.numpy(), q.double().numpy(), cu, lens, tables.numpy(), 128 ** -0.5)
    ref, ref_lse = int8_ref.attention(*args)
    # a score is off by (2^-10 + 2^-11) sum |q||k| scale more (factor and product rounded), a value by as much of itself
    kmax = 127 * 0.051
    more = 2 * (1.5 * 2.0 ** -10) * np.abs(q.double().numpy()).sum(2).max() * kmax * 128 ** -0.5 + 1.5 * 2.0 ** -10
    err, err_lse = bounds(*args, ref, 2.0 ** -11 + more, weight_abs=2.0 ** -32)
    check(out, None, ref, ref_lse, err, err_lse)
    assert np.abs(out.double().cpu().numpy() - ref).max() < 4e-3 * np.abs(ref).max()


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("bs", [8, 16])
def test_larger_scales_behind_a_row_block(bs, kv):
    """Pages in the last key tile of a causal row block that none of its rows sees, with scales 2^14 times those before."""
    lens, d = [552], 128                                       # rows 0-255 see keys up to 295, in the tile of keys 256-383
    codes, scales = pool(-(-552 // bs) + 2, 1, bs, d, 21, 1)
    tables = tables_of(lens, bs, codes.shape[0], -(-552 // bs) + 1, 21)
    for i in range(-(-552 // bs)):
        scales[tables[0, i], kv] = 2.0 ** (4 if i * bs >= 304 else -10)
    run(lens, [512], 2, 1, d, bs, "f16", 21, codes=codes, scales=scales, scale=0.01)


def test_scale_zero_and_below():
    run([200], [150], 2, 1, 64, 16, "f16", 11, scale=0.0)
    run([200], [150], 2, 1, 64, 16, "f16", 11, scale=-0.125)


@pytest.mark.parametrize("first", [-100, 0])
def test_small_weights_add_up(first):
    """One key far above 30000 others, each of whose weights alone is below f16's range, with a value of its own and without."""
    d, bs, n = 64, 64, 30016
    codes = torch.zeros((n // bs, 2, 1, bs, d), dtype=torch.int8)
    codes[:, 1] = 100
    codes[0, 0, 0, 0], codes[0, 1, 0, 0] = 64, first
    scales = torch.ones((n // bs, 2, 1)) / 64
    tables = torch.arange(n // bs, dtype=torch.int32)[None]
    q = torch.full((2, 1, d), 18.0 / d).half()
    out = pkv.paged_attn_prefill(codes.cuda(), q.cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda(),
                                 torch.tensor([n], dtype=torch.int32).cuda(), tables.cuda(), max_q_len=2, scale=1.0,
                                 out_dtype=torch.float32, scales=scales.cuda())
    rest = (n - 1) * np.exp(-float(q[0, 0, 0]) * d)
    want = (100 * rest + first) / 64 / (rest + 1)
    # A weight of 2^-26 is 2^-19 in the product, off by half of f16's 2^-24 there: 2^-6 of itself. The tensor core aligns
    # the 16 products of a step to its accumulator and truncates: a product loses at most 2^-23 of the accumulator, here
    # of |first| / 64 (its largest part), so n products at most n 2^-23 |first| / 64.
    bound = rest * 100 / 64 * 2.0 ** -6 * 1.1 + n * 2.0 ** -23 * abs(first) / 64
    assert abs(out[1, 0, 0].item() - want) <= bound, (out[1, 0, 0].item(), want)


def test_what_is_not_a_number():
    """Rows that see a key of a page whose scale is not finite are NaN; rows before it in the same tile are not."""
    codes, scales = pool(8, 1, 16, 64, 3)
    q = torch.randn((100, 2, 64), generator=torch.Generator().manual_seed(1)).half()
    tables = torch.tensor([[4, 2, 0, 1, 3, 5, 6]], dtype=torch.int32)
    clean = scales.clone()
    for kv, value in ((0, float("nan")), (1, float("nan")), (1, float("inf"))):
        scales = clean.clone()
        scales[1, kv] = value                                  # positions 48 .. 63
        scales[6] = float("nan")                               # behind what any row sees
        lse = torch.empty((96, 2), device="cuda")
        call = lambda s, n, **kw: pkv.paged_attn_prefill(codes.cuda(), q[:n].cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                                                         torch.tensor([n], dtype=torch.int32).cuda(), tables.cuda(), max_q_len=n,
                                                         scales=s.cuda(), **kw)
        out = call(scales, 96, lse=lse)
        assert torch.isfinite(out[:48]).all() and torch.isnan(out[48:96]).all()
        assert torch.equal(out[:48], call(torch.nan_to_num(scales, nan=1.0, posinf=1.0) * 0 + clean, 96)[:48])
        assert torch.isfinite(lse[:48]).all() and torch.isnan(lse[48:96]).all() == (kv == 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,heads,new", [(2, 1, [1, 127, 128]), (8, 2, [64, 63]), (8, 2, [65, 3]), (6, 1, [50, 128]), (5, 1, [9]),
                                          (16, 1, [16, 1, 5]), (40, 1, [31, 32]), (64, 1, [4, 3, 2]), (128, 1, [2, 1]),
                                          (256, 1, [1, 1]), (24, 2, [20, 21]), (12, 4, [100])])
def test_short_chunks(hq, heads, new, d):
    """Rows of several heads in one block: every number of heads that a block takes, blocks of one tile and of two."""
    run([n + 37 * i + 5 for i, n in enumerate(new)], new, hq, heads, d, 16, "bf16", hq + new[0])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq", [1, 2, 3, 5, 11, 17])
@pytest.mark.parametrize("lens,new", [([3000], [200]), ([2100, 1, 300], [20, 1, 300]), ([1500, 1400], [130, 256])])
def test_blocks_shared_by_several_ctas(lens, new, hq, causal):
    """Few blocks over long contexts, from 2 to 8 CTAs a block; some of them without a key of theirs, or with masked ones only."""
    run(lens, new, hq, hq, 64, 16, "f16", hq, causal=causal)


@pytest.mark.parametrize("hq,heads,d,bs", [(8, 2, 128, 8), (4, 1, 128, 512), (32, 2, 64, 64), (16, 16, 128, 128)])
def test_shared_blocks_of_short_chunks(hq, heads, d, bs):
    run([4000, 700, 2500], [33, 5, 64], hq, heads, d, bs, "bf16", bs)
    run([4000, 700, 2500], [33, 1, 64], hq, heads, d, bs, "bf16", bs, mixed=True)


@pytest.mark.parametrize("kv", [0, 1])
def test_not_a_number_in_a_shared_block(kv):
    """Only the rows that see the page are NaN, whichever CTA had it; pages behind the last key do not count."""
    d, bs, n, new = 128, 16, 3000, 250
    codes, scales = pool(200, 1, bs, d, 5)
    tables = torch.randperm(200, generator=torch.Generator().manual_seed(2))[:190].to(torch.int32)[None]
    q = torch.randn((new, 4, d), generator=torch.Generator().manual_seed(3)).half()

    def call(s):
        lse = torch.empty((new, 4), device="cuda")
        out = pkv.paged_attn_prefill(codes.cuda(), q.cuda(), torch.tensor([0, new], dtype=torch.int32).cuda(),
                                     torch.tensor([n], dtype=torch.int32).cuda(), tables.cuda(), max_q_len=new, lse=lse,
                                     scales=s.cuda())
        assert pkv.get_device_error() == 0
        return out, lse

    want, want_lse = call(scales)
    for page, value in ((181, float("nan")), (3, float("inf")), (188, float("nan"))):
        s = scales.clone()
        s[tables[0, page], kv] = value
        out, lse = call(s)
        first = min(new, max(0, page * bs - (n - new)))        # the first row that sees it
        assert torch.equal(out[:first], want[:first]) and torch.isnan(out[first:]).all()
        assert torch.equal(lse[:first], want_lse[:first])
        assert torch.isnan(lse[first:]).all() if kv == 0 else torch.equal(lse[first:], want_lse[first:])


def test_shared_blocks_again_and_again():
    """The same bits from call to call, in a graph too."""
    codes, scales = pool(130, 2, 16, 128, 6)
    i = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    tables = torch.randperm(130, generator=torch.Generator().manual_seed(2))[:128].to(torch.int32).reshape(1, 128).cuda()
    q = torch.randn((300, 4, 128), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    call = lambda: pkv.paged_attn_prefill(codes, q, i_cu, i_len, tables, max_q_len=300, scales=scales)
    codes, scales, i_cu, i_len = codes.cuda(), scales.cuda(), i([0, 300]), i([2040])
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(20):
        graph.replay()
        assert torch.equal(out, want) and torch.equal(call(), want)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("lens,new,hq", [([3000], [200], 2), ([300], [300], 40)])
def test_largest_values(lens, new, hq):
    """Values whose sum over the context is within FP32: blocks of one CTA and of several."""
    d, bs = 64, 16
    codes, scales = pool(200, 1, bs, d, 31)
    codes[:, 1], scales[:, 1] = codes[:, 1].abs().clamp(min=100), 2.0 ** 107
    run(lens, new, hq, 1, d, bs, "bf16", 31, codes=codes, scales=scales, scale=0.001)


def test_bad_arguments_are_flagged():
    codes, scales = pool(8, 1, 16, 64, 3)
    q = torch.randn((20, 1, 64)).half().cuda()
    i = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    call = lambda lens, t: pkv.paged_attn_prefill(codes.cuda(), q, i(0, 10, 20), lens, t, max_q_len=10, scales=scales.cuda())
    out = call(i(20, 20), i([0, 9], [2, 1]))
    assert pkv.get_device_error() == 5 and torch.isfinite(out[10:]).all()
    call(i(9, 20), i([0, 3], [2, 1]))
    assert pkv.get_device_error() == 5
    call(i(20, 33), i([0, 3], [2, 1]))
    assert pkv.get_device_error() == 5


def test_mixed():
    """Decode rows, chunks, empty sequences in one call."""
    run([300, 45, 700, 129, 33], [1, 45, 200, 1, 5], 8, 2, 128, 16, "bf16", 21, mixed=True)
    run([300, 45], [1, 1], 4, 4, 64, 32, "f16", 22, mixed=True)


def test_append_then_attend_and_in_a_graph():
    """Prompt chunks appended and attended, then decode steps, then a fork: as a server runs them, against the reference."""
    d, bs, heads, hq = 128, 16, 2, 8
    g = torch.Generator().manual_seed(1)
    codes = torch.zeros((64, 2, heads, bs, d), dtype=torch.int8, device="cuda")
    scales = torch.zeros((64, 2, heads), device="cuda")
    tables = torch.arange(40, dtype=torch.int32).reshape(2, 20)
    rc, rs = codes.cpu().numpy().copy(), scales.cpu().numpy().copy()
    ctx, scale = [0, 0], d ** -0.5
    i = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32).cuda()
    t = tables.cuda()
    for new in ([130, 77], [60, 1], [1, 90]):
        cu = np.concatenate(([0], np.cumsum(new)))
        q, k, v = (torch.randn((sum(new), h, d), generator=g).bfloat16() for h in (hq, heads, heads))
        pkv.kv_cache_append(codes, k.cuda(), v.cuda(), i(cu), i(ctx), t, scales=scales)
        int8_ref.append(rc, rs, k.double().numpy(), v.double().numpy(), cu.tolist(), ctx, tables.numpy())
        ctx = [a + b for a, b in zip(ctx, new)]
        out = pkv.paged_attn_mixed(codes, q.cuda(), i(cu), i(ctx), t, max_q_len=max(new), scales=scales)
        args = (rc, rs, q.double().numpy(), cu, ctx, tables.numpy(), scale)
        ref, ref_lse = int8_ref.attention(*args)
        check(out, None, ref, ref_lse, *bounds(*args, ref, 2.0 ** -11, weight_abs=2.0 ** -32))
    # four children of two parents
    ft, fl = pkv.kv_cache_fork(codes, t, i(ctx), i([0, 0, 1, 1]), i([40, 41, 42, -1]), scales=scales)
    q, k, v = (torch.randn((4, h, d), generator=g).bfloat16().cuda() for h in (hq, heads, heads))
    graph = torch.cuda.CUDAGraph()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    spare, spare_s = codes.clone(), scales.clone()
    with torch.cuda.stream(warm):
        pkv.paged_attn_decode_step(spare, q, ft, fl, k, v, scales=spare_s)
    torch.cuda.current_stream().wait_stream(warm)
    with torch.cuda.graph(graph):
        out = pkv.paged_attn_decode_step(codes, q, ft, fl, k, v, scales=scales)
    fold = int8_ref.fork([(rc, 3), (rs, None)], tables.numpy(), ctx, [0, 0, 1, 1], [40, 41, 42, -1], bs)
    assert np.array_equal(ft.cpu().numpy(), fold[0])
    graph.replay()
    args = (rc, rs, q.double().cpu().numpy(), np.arange(5), fold[1].tolist(), fold[0], scale)
    ref, ref_lse = int8_ref.attention(*args, causal=False)
    check(out, None, ref, ref_lse, *bounds(*args, ref, 2.0 ** -21, causal=False))
    int8_ref.append(rc, rs, k.double().cpu().numpy(), v.double().cpu().numpy(), list(range(5)), fold[1].tolist(), fold[0])
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    assert pkv.get_device_error() == 0
