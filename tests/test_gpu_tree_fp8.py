"""paged_attn_tree over an FP8 cache, against the definition in 64 bits over the dequantised values."""
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Fp8Case(Case):
    """The same inputs with the cache as E4M3 codes and row scales; self.cache holds the values they stand for."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        x = self.cache.float()
        self.scales = (x.abs().amax(-1) / 448.0).contiguous()
        self.codes = (x / self.scales[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.refresh()

    def refresh(self):
        self.cache = self.codes.view(torch.float8_e4m3fn).double() * self.scales.double()[..., None]

    def run(self, **kw):
        dev = {k: getattr(self, k).cuda() for k in ("codes", "scales", "q", "mask", "cu", "table")}
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        out = pkv.paged_attn_tree(dev["codes"], dev["q"], dev["mask"], dev["cu"], lens, dev["table"], max_q_len=self.max_q,
                                  lse=lse, scales=dev["scales"], **kw)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def p_half(self, dtype):
        """Each weight, times what its value's row scale is above a power of two, is rounded once to the cache's 16-bit
        type: half a step of it. The values' codes times those powers are exact."""
        return torch.finfo(self.dt).eps / 2


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (128, 8), (128, 128), (64, 512)])
def test_one_small_tree(d, bs, dtype):
    c = Fp8Case([100], [9], 8, 2, d=d, bs=bs, dtype=dtype, seed=d + bs)
    c.check(c.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n", [(4, 4, 1), (4, 4, 129), (4, 4, 300), (8, 2, 33), (8, 2, 64), (6, 2, 43), (32, 1, 5),
                                      (131, 1, 2), (40, 4, 31)])
def test_groups_and_row_blocks(hq, hkv, n, d):
    c = Fp8Case([n + 333, n, n + 5], [n, n, max(1, n // 2)], hq, hkv, d=d, seed=hq + n)
    c.check(c.run(), (hq, hkv, n))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_ragged_batch(d, dtype):
    lens = [1, 2, 127, 128, 129, 1, 700, 1500, 64, 257, 300, 2047]
    nodes = [1, 2, 3, 64, 65, 0, 31, 17, 64, 1, 40, 63]
    c = Fp8Case(lens, nodes, 8, 2, d=d, bs=16, dtype=dtype, seed=d)
    c.check(c.run())


@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts(d):
    c = Fp8Case([20011], [7], 4, 1, d=d, bs=64, seed=1)
    c.check(c.run())
    c = Fp8Case([9000, 5000, 12000], [40, 64, 3], 8, 2, d=d, bs=32, seed=2)
    c.check(c.run())
    c = Fp8Case([4000, 130], [70, 70], 8, 2, d=d, bs=16, seed=3, masks="any")
    out, lse = c.run(out_dtype=torch.float32)
    c.check((out, lse))


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("d,hq", [(64, 4), (128, 4), (128, 16)])
def test_what_is_masked_may_hold_anything(bad, d, hq):
    """Scales that are not finite: of nodes that only some see, behind the context, in pages not listed."""
    n = 40
    c = Fp8Case([150, n], [n, n], hq, 2, d=d, seed=9, masks="any")
    c.codes[(c.codes & 0x7F) == 0] += 1    # (0 times infinity is left to the other test)
    for b, L in enumerate(c.lens):
        for i in range(n):
            for j in (3, 38):
                if i != j and i % 3:
                    c.hide(b, i, j)
        for pos in range(L, -(-L // c.bs) * c.bs):
            p, o = c.slot(b, pos)
            c.scales[p, :, :, o] = bad
            c.codes[p, :, :, o] = 0x7F
        p, o = c.slot(b, L - n + 3)
        c.scales[p, 1, :, o] = bad
        p, o = c.slot(b, L - n + 38)
        c.scales[p, 1, 0, o] = bad
    used = set(c.table[c.table >= 0].tolist())
    for p in set(range(c.codes.shape[0])) - used:
        c.scales[p] = bad
    c.refresh()
    out, lse = c.run()
    c.check((out, lse))
    ro, _, _ = c.exact()
    assert torch.equal(out.isnan(), ro.isnan())
    inf = ro.isinf()
    assert torch.equal(out[inf].double(), ro[inf])
    # a node that nobody else sees: everything of it
    c = Fp8Case([150], [n], hq, 2, d=d, seed=10)
    for i in range(n):
        c.hide(0, i, 11)
    p, o = c.slot(0, 150 - n + 11)
    c.scales[p, :, :, o] = bad
    c.codes[p, :, :, o] = 0x7F
    c.refresh()
    c.check(c.run())


def test_after_append_it_agrees_with_the_prefill():
    """A chain is the causal chunk that paged_attn_prefill attends over the same cache."""
    from paged_kv_flash_cache_gb300 import workloads as W
    n = 24
    c = Fp8Case([500, n + 7], [n, n], 8, 2, seed=18)
    c.mask = W.tree_mask([list(range(-1, n - 1))] * 2)
    c.sees = [torch.ones((n, n), dtype=torch.bool).tril()] * 2
    c.check(c.run())
    out, _ = c.run(out_dtype=torch.float32)
    ref = pkv.paged_attn_prefill(c.codes.cuda(), c.q.cuda(), c.cu.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(),
                                 c.table.cuda(), max_q_len=n, out_dtype=torch.float32, scales=c.scales.cuda())
    # values rounded to bf16 here (half a step, 2^-8), P to f16 there (2^-11)
    assert (out - ref.cpu()).abs().max() <= (2.0 ** -8 + 2.0 ** -10) * float(c.cache.abs().max())


@pytest.mark.parametrize("dtype,factor", [("bf16", 2.0 ** -90), ("bf16", 1e-20), ("bf16", 1e30), ("bf16", 0.3), ("f16", 2.0 ** -12),
                                          ("f16", 3e-3), ("f16", 4000.0)])
@pytest.mark.parametrize("d,n", [(64, 20), (128, 20), (128, 70)])
def test_value_scales_of_any_size(d, n, dtype, factor):
    """The value rows' scales, each row's its own, far from 1; some rows of zeros with a scale of 0."""
    c = Fp8Case([300, n + 1], [n, n], 4, 2, d=d, seed=19, dtype=dtype)
    g = torch.Generator().manual_seed(20)
    c.scales[:, 1] *= factor * torch.rand(c.scales[:, 1].shape, generator=g)
    zero = torch.rand(c.scales[:, 1].shape, generator=g) < 0.1
    c.scales[:, 1][zero] = 0.0
    c.codes[:, 1][zero] = 0
    c.refresh()
    out, _ = c.run(out_dtype=torch.float32)
    ro, _, vmax = c.exact()
    # as check(): FP32 sums of both products and ex2, and half a step of the cache's type on each weight
    tol = (2 * (0.9 * d ** 1.5 * 2.0 ** -24 + 2.0 ** -17) + c.p_half(out.dtype)) * vmax
    assert vmax > 0 and (out.double() - ro).abs().max() <= tol
    assert pkv.get_device_error() == 0
