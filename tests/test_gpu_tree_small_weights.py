"""Many keys whose weights are far below the largest one: each is small, their sum is not."""
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,n,hq", [(64, 1, 4), (128, 5, 4), (128, 70, 4), (256, 5, 2)])
@pytest.mark.parametrize("gap", [12.0, 17.5, 20.0])
def test_one_key_far_above_the_others(d, n, hq, dtype, fp8, gap):
    """The first token's score is `gap` above everyone else's (equal) ones, its value 0, the others' values 1: the output is
    S / (1 + S) with S = (L - 1) e^-gap, the weights of the others in full. Enough sequences (over the same pages) that an
    item is not split over many runs, of which only the first would see the large weight."""
    if fp8 and d == 256:
        pytest.skip("an FP8 cache has head_dim 64 or 128")
    dt, L, bs, batch = DT[dtype], 30001, 64, 304
    pages = -(-L // bs)
    # q . k: the first token's along q, the others' 0; gap in units that both types and E4M3 (of a row's maximum) hold exactly
    q = torch.full((batch * n, hq, d), 1.0, dtype=dt, device="cuda")
    kv = torch.zeros((pages, 2, 1, bs, d), dtype=dt, device="cuda")
    kv[:, 1] = 1.0
    kv[0, 0, 0, 0] = 1.0
    kv[0, 1, 0, 0] = 0.0
    scale = gap / d
    cache, scales = kv, None
    if fp8:
        scales = (kv.float().abs().amax(-1) / 448.0).contiguous()
        cache = torch.where(kv != 0, 448.0, 0.0).to(torch.float8_e4m3fn)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1)
    lens = torch.full((batch,), L, dtype=torch.int32, device="cuda")
    mask = W.tree_mask([list(range(-1, n - 1))] * batch).cuda()
    seen = torch.arange(L - n + 1, L + 1, dtype=torch.float64).repeat(batch)   # node i sees the context and i + 1 nodes
    s = (seen - 1) * math.exp(-gap)
    ref, ref_lse = s / (1 + s), gap + torch.log1p(s)
    for out_dtype in (dt, torch.float32):
        lse = torch.empty((batch * n, hq), device="cuda")
        out = pkv.paged_attn_tree(cache, q, mask, W.cu_lens([n] * batch).cuda(), lens, table, max_q_len=n, scale=scale,
                                  out_dtype=out_dtype, lse=lse, scales=scales).double().cpu()
        # Each weight: half a step of its 16 bits where it is rounded once, else FP32's (ex2, scores: see the tree tests);
        # f16 has no step below 2^-24, and the weights are 2^4 (FP8) or 2^7 times themselves there: half of it for each key.
        once = torch.finfo(dt).eps / 2 if fp8 or (n * hq > 128 and d <= 128 and out_dtype != torch.float32) else 0.0
        flat = (L * 2.0 ** -25 / (2.0 ** 4 if fp8 else 2.0 ** 7)) if dtype == "f16" else 0.0
        rel = 2 * (gap * d * 2.0 ** -24 + 2.0 ** -17) + once
        tol = rel * ref + flat + torch.finfo(out_dtype).eps / 2 * ref
        assert ((out - ref[:, None, None]).abs() <= tol[:, None, None]).all(), (float(out.max()), float(ref.max()))
        assert ((lse.cpu().double() - ref_lse[:, None]).abs() <= gap * d * 2.0 ** -24 + 2.0 ** -20 * (1 + gap)).all()
    assert pkv.get_device_error() == 0
