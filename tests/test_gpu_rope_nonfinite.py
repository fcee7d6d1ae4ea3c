"""Infinities and NaN through rope_append: what a row that holds one leaves in q_out and in the pages."""
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_rope import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def put(c, token, which, head, elements, bad):
    """`bad` into elements of one head row of q, k or v; the others stay."""
    base = {"q": 0, "k": c.hq, "v": c.hq + c.hkv}[which] + head
    for e in elements:
        c.x[token, base * c.d + e] = bad


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_fp8_rows(d, inter, norm, bad):
    """One scale stands for a row, so a row with a NaN or an infinity is one that is not finite: its scale says so, and no
    element of it reads as a number. Every other row is what it is without them."""
    c = Case([9, 5], [3, 40], 4, 4, d=d, rot=d // 2, fp8=True, inter=inter, norm=norm, seed=d, dtype="bf16")
    good = c.run()
    hit = [(1, "k", 0, [5]), (2, "k", 3, range(d)), (3, "v", 1, [d - 1]), (4, "v", 2, range(d)), (10, "k", 1, [d - 1, 0]),
           (10, "v", 1, [7]), (13, "v", 3, [d // 2])]
    for token, which, head, elements in hit:
        put(c, token, which, head, elements, bad)
    out, cache, scales = c.run()
    where = list(c.rows())
    mine = torch.zeros_like(scales, dtype=torch.bool)
    for token, which, head, _ in hit:
        p, o = where[token]
        mine[p, int(which == "v"), head, o] = True
    value = cache.view(torch.float8_e4m3fn).float() * scales[..., None]
    assert not scales[mine].isfinite().any()
    assert not value[mine].isfinite().any()
    if math.isnan(bad):
        assert scales[mine].isnan().all()
    assert torch.equal(scales[~mine], good[2][~mine]) and torch.equal(cache[~mine], good[1][~mine])
    assert torch.equal(out, good[0])
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 128), (256, 64)])
def test_16_bit_rows_and_queries(d, rot, inter, norm, bad):
    """Element by element what the formulas give."""
    c = Case([9, 5], [3, 40], 4, 2, d=d, rot=rot, inter=inter, norm=norm, seed=d, dtype="f16")
    for token, which, head, elements in ((1, "k", 0, [5]), (2, "q", 3, range(d)), (3, "v", 1, [d - 1]), (4, "q", 2, [d - 1]),
                                         (10, "k", 1, [0, d - 1]), (12, "q", 0, [rot // 2])):
        put(c, token, which, head, elements, bad)
    out, cache, _ = c.run()
    q, k, v = c.views(c.x)
    page, off = (torch.tensor([w[i] for w in c.rows()], dtype=torch.long) for i in (0, 1))
    for got, ref in ((out, c.turned(q, c.qw)), (cache[page, 0, :, off], c.turned(k, c.kw)), (cache[page, 1, :, off], v.double())):
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.isinf(), ref.isinf())
        assert torch.equal(got[got.isinf()].double(), ref[ref.isinf()])
    assert pkv.get_device_error() == 0
