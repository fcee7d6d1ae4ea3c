"""kv_cache_compact of lists of very different lengths in one call: the launch goes by their average."""
import pytest
import torch

from tests.test_gpu_compact import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("others,rows", [(1, 1000), (0, 700), (8, 3000)])
def test_one_long_list_among_short_ones(others, rows, d, fp8):
    g = torch.Generator().manual_seed(rows + d)
    batch, long_one = 64, 41
    keep, start, lens = [], [], []
    for b in range(batch):
        n = rows if b == long_one else others
        first = int(torch.randint(0, 40, (1,), generator=g))
        span = 2 * n + 20
        at = torch.randperm(span, generator=g)[:n].sort().values + first
        keep.append(at.tolist())
        start.append(first)
        lens.append(first + span)
    Case(keep, start, lens, hkv=2, d=d, fp8=fp8, seed=rows).check()
