"""A token whose cached K or V holds a NaN or an infinity, verified (paged_attn_tree) and decoded (paged_attn_decode): the
two have to agree on what is not finite, whichever call wrote the token."""
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def filled(lens, hkv, d, bs, dt, fp8, k, v, by_rope):
    """A cache with the sequences' k and v [sum lens, Hkv, D] written by rope_append (nothing rotated) or kv_cache_append."""
    need = [-(-n // bs) for n in lens]
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 1
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    table = table.cuda()
    shape = (at, 2, hkv, bs, d)
    cache = torch.zeros(shape, dtype=torch.uint8 if fp8 else dt, device="cuda")
    scales = torch.zeros(shape[:4], device="cuda") if fp8 else None
    cu, zero = W.cu_lens(lens).cuda(), torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    if by_rope:
        pkv.rope_append(cache, k, k, v, torch.empty(0, device="cuda"), cu, zero, table,
                        positions=torch.zeros(k.shape[0], dtype=torch.int32, device="cuda"), scales=scales)
    else:
        pkv.kv_cache_append(cache, k, v, cu, zero, table, scales=scales)
    return cache, scales, table


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("by_rope", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(4, 4, 128, "f16"), (8, 2, 128, "bf16"), (8, 2, 64, "f16"), (8, 2, 64, "bf16")])
def test_tree_and_decode_agree(hq, hkv, d, dtype, fp8, by_rope, bad):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(hq + d)
    lens = [70, 300, 129, 40, 33, 200]
    k, v = (torch.randn((sum(lens), hkv, d), generator=g).to(dt) for _ in range(2))
    q = torch.randn((len(lens), hq, d), generator=g).to(dt).cuda()
    first = [0] + torch.tensor(lens).cumsum(0).tolist()
    k[first[0] + 3, 0, 5] = bad                  # an element of K in the context
    v[first[1] + 250, 1, 7] = bad                # of V
    v[first[2] + 128, 0, d - 1] = bad            # of V of the last token, which is the tree's node
    k[first[3] + 20, 1] = bad                    # a row of K
    v[first[4] + 10, 0] = bad                    # a row of V
    k[first[5] + 199, 0, 0] = bad                # of K of the node
    cache, scales, table = filled(lens, hkv, d, 16, dt, fp8, k.cuda(), v.cuda(), by_rope)
    n_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    mask = torch.ones((len(lens), 1), dtype=torch.int32, device="cuda")
    for out_dtype in (dt, torch.float32):
        tree = pkv.paged_attn_tree(cache, q, mask, W.cu_lens([1] * len(lens)).cuda(), n_lens, table, max_q_len=1,
                                   out_dtype=out_dtype, scales=scales)
        step = pkv.paged_attn_decode(cache, q, table, n_lens, out_dtype=out_dtype, scales=scales)
        # (of an infinity that is seen either may make a NaN: P in two parts, of which one is 0 or negative)
        assert torch.equal(tree.isfinite(), step.isfinite())
        if math.isnan(bad):
            # by the definition: a NaN in K makes its heads NaN, one in V its column (one scale a row: rope_append its row)
            want = torch.zeros((len(lens), hkv, hq // hkv, d), dtype=torch.bool)
            want[0, 0], want[5, 0] = True, True
            if not (fp8 and not by_rope):        # (kv_cache_append stores an FP8 row that is all NaN as zeros)
                want[3, 1], want[4, 0] = True, True
            if fp8 and by_rope:
                want[1, 1], want[2, 0] = True, True
            else:
                want[1, 1, :, 7], want[2, 0, :, d - 1] = True, True
            assert torch.equal(tree.cpu().isnan(), want.reshape(len(lens), hq, d))
        # finite ones: P in 16 bits on either side, each half a step of max |v|, and the output's own rounding
        fin = tree.isfinite()
        vmax = float(v[v.isfinite()].abs().max())
        step_of = torch.finfo(dt).eps / 2
        assert (tree.double() - step.double()).abs()[fin].max() <= (4 * step_of + 2.0 ** -12) * vmax
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,hq", [(64, 4), (128, 4), (128, 16)])
def test_nan_codes_where_some_do_not_see_them(d, hq, dtype):
    """NaN codes under finite scales, of context, of nodes that only some see, behind the end: NaN for those that see them."""
    from tests.test_gpu_tree_fp8 import Fp8Case
    n = 40
    c = Fp8Case([150, n, 700], [n, n, n], hq, 2, d=d, dtype=dtype, seed=9, masks="any")
    for b, L in enumerate(c.lens):
        for i in range(n):
            for j in (3, 21, 38):
                if i != j and i % 3:
                    c.hide(b, i, j)
        for pos in range(L, -(-L // c.bs) * c.bs):
            p, o = c.slot(b, pos)
            c.codes[p, :, :, o] = 0x7F
        p, o = c.slot(b, L - n + 3)
        c.codes[p, 1, :, o] = 0xFF
        p, o = c.slot(b, L - n + 38)
        c.codes[p, 1, 0, o, 5] = 0x7F
        c.codes[p, 1, 1, o, d - 1] = 0xFF
        p, o = c.slot(b, L - n + 21)
        c.codes[p, 0, 1, o, 17] = 0x7F           # K
    p, o = c.slot(2, 130)
    c.codes[p, 1, 0, o, 9] = 0xFF                # context
    c.refresh()
    for out_dtype in (None, torch.float32):
        out, lse = c.run(out_dtype=out_dtype)
        ro, rl, vmax = c.exact()
        assert torch.equal(out.isnan(), ro.isnan()) and torch.equal(lse.isnan(), rl.isnan())
        assert ro.isnan().any() and ro.isfinite().any()
        fin = ro.isfinite()
        tol = (2 * (0.9 * d ** 1.5 * 2.0 ** -24 + 2.0 ** -17) + c.p_half(out.dtype)) * vmax
        assert ((out.double() - ro).abs()[fin] <= tol + torch.finfo(out.dtype).eps / 2 * 1.01 * ro.abs()[fin] + 1e-7).all()
    assert pkv.get_device_error() == 0
