"""paged_attn_tree over runs of many short items: the lanes of a narrow block hand their (max, sum) over item after item,
with nothing else between them that would wait."""
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests.test_gpu_tree import Case
from tests.test_gpu_tree_fp8 import Fp8Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def short(cls, d, most, big=0, **kw):
    """200 sequences of 8 KV heads: about ten items a CTA, each of one or two key tiles; `big` of them in wide blocks."""
    g = torch.Generator().manual_seed(d + most)
    lens = torch.randint(1, most, (200,), generator=g).tolist()
    nodes = [min(L, int(torch.randint(1, 8, (1,), generator=g))) for L in lens]
    for b in range(big):
        lens[7 * b], nodes[7 * b] = max(lens[7 * b], 70), 70
    # scores far apart, so that an item's (max, sum) is not its neighbour's
    c = cls(lens, nodes, 16, 8, d=d, seed=most, **kw)
    c.q = (c.q.float() * torch.rand((c.q.shape[0], 1, 1), generator=g) * 2).to(c.dt)
    return c


@pytest.mark.parametrize("cls", [Case, Fp8Case])
@pytest.mark.parametrize("d,most,big", [(64, 120, 0), (128, 120, 0), (128, 250, 0), (64, 250, 12), (128, 60, 12)])
def test_many_short_items_a_run(cls, d, most, big):
    c = short(cls, d, most, big)
    first = c.run(out_dtype=torch.float32)
    # scores up to twice the size that check() counts with: its bound on them, twice
    ro, rl, vmax = c.exact()
    rel = 2 * 0.9 * d ** 1.5 * 2.0 ** -24
    tol = 2 * (rel + 2.0 ** -17) * vmax + c.p_half(torch.float32) * vmax
    assert ((first[0].double() - ro).abs() <= tol + 1e-7).all()
    assert ((first[1].double() - rl).abs() <= rel + 2.0 ** -20 * (1 + rl.abs())).all()
    for _ in range(20):
        again = c.run(out_dtype=torch.float32)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert pkv.get_device_error() == 0
