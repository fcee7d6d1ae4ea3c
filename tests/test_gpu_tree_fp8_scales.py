"""paged_attn_tree over FP8 caches whose value scales lie at the ends of what the split into a power of two and the rest takes."""
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_tree_fp8 import Fp8Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dtype,low", [("f16", -33), ("f16", -23), ("f16", -22), ("f16", -17), ("f16", -16), ("f16", -15), ("f16", 6),
                                       ("f16", 7), ("f16", 8), ("f16", 9), ("bf16", -126), ("bf16", -101), ("bf16", 7), ("bf16", 8),
                                       ("bf16", 12), ("bf16", 60), ("bf16", 110)])
@pytest.mark.parametrize("d,n", [(64, 20), (128, 20), (128, 70)])
def test_value_scales_at_the_ends(d, n, dtype, low):
    """Every value row's scale between 2^low and 2^(low + 1), scores far apart. f16 takes value scales below 2^10, and rounds values
    below 2^-15 times a code's step (2^-9) as subnormals: by 2^-25 of what is left of the scale."""
    c = Fp8Case([300, n + 1], [n, n], 4, 2, d=d, seed=19, dtype=dtype)
    g = torch.Generator().manual_seed(low + 200)
    c.q = (c.q.float() * 4).to(c.dt)
    c.scales[:, 1] = 2.0 ** low * (1 + torch.rand(c.scales[:, 1].shape, generator=g) * 0.999)
    c.refresh()
    out, _ = c.run(out_dtype=torch.float32)
    ro, _, vmax = c.exact()
    # Fp8Case.check()'s bound, scores four times as large; values as above, where e = low is held to [-22, 7]
    step = 2.0 ** -25 * 2.0 ** (low + 1 - max(low, -22)) if dtype == "f16" and low < -15 else 0.0
    tol = (2 * (4 * 0.9 * d ** 1.5 * 2.0 ** -24 + 2.0 ** -17) + c.p_half(out.dtype)) * vmax + step
    if dtype == "f16" and low < -22:
        # rest below 1: 2^4 rest w loses what is below 2^-25, for at most 320 keys
        tol += 320 * 2.0 ** -25 / 2 ** 4 * 448 * 2.0 ** -22
    assert vmax > 0 and out.isfinite().all() and (out.double() - ro).abs().max() <= tol
    assert pkv.get_device_error() == 0
