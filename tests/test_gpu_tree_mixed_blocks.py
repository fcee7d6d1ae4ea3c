"""Trees over an FP8 cache whose runs go from narrow row blocks to wide ones and back: many calls, each with its results and
the device's error word (the conversion of a wide block's first keys once overtook a narrow block's last values)."""
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hq", [(70, 4), (33, 4), (97, 2)])
def test_wide_and_narrow_blocks_in_turn(n, hq):
    d, bs, batch, length = 128, 64, 304, 12001
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = -(-length // bs)
    cache = (torch.randn((pages, 2, 1, bs, d), generator=g, device="cuda") * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.rand((pages, 2, 1, bs), generator=g, device="cuda") * 0.02 + 0.002
    q = torch.randn((n, hq, d), generator=g, device="cuda").half().repeat(batch, 1, 1)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(batch, 1)
    lens = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    mask, cu = W.tree_mask([list(range(-1, n - 1))] * batch).cuda(), W.cu_lens([n] * batch).cuda()
    # two cuts of the same keys: each weight rounded once to f16 on either side (half a step, 2^-11) times values of at most
    # vmax, and the output's rounding
    vmax = float(448 * scales.max())
    tol = 2 * 2.0 ** -11 * vmax + torch.finfo(torch.float16).eps * vmax
    first = None
    for _ in range(60):
        out = pkv.paged_attn_tree(cache, q, mask, cu, lens, table, max_q_len=n, scales=scales)
        assert pkv.get_device_error() == 0
        # every sequence is the same one, and its runs are cut alike
        out = out.reshape(batch, n, hq, d)
        assert torch.isfinite(out).all()
        first = out[0].clone() if first is None else first
        assert (out.float() - first.float()).abs().max() <= tol
