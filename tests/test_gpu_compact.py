"""kv_cache_compact on the GPU: the cache's bits against the same moves made one by one on the host."""
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Case:
    """keep: a list of positions for each sequence; start: where they go; lens: tokens each table holds."""

    def __init__(self, keep, start, lens, hkv=2, d=128, bs=16, fp8=False, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.keep, self.start, self.bs = keep, start, bs
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + 2
        order = torch.randperm(nb, generator=g).tolist()
        self.table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
            at += k
        shape = (nb, 2, hkv, bs, d)
        if fp8:
            self.cache = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
            self.scales = torch.rand(shape[:4], generator=g)
        else:
            self.cache = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16).view(torch.bfloat16)
            self.scales = None

    def args(self):
        flat = [p for k in self.keep for p in k]
        return (torch.tensor(flat, dtype=torch.int32).cuda(), W.cu_lens([len(k) for k in self.keep]).cuda(),
                torch.tensor(self.start, dtype=torch.int32).cuda(), self.table.cuda())

    def run(self, **kw):
        cache = self.cache.cuda()
        scales = None if self.scales is None else self.scales.cuda()
        pkv.kv_cache_compact(cache, *self.args(), scales=scales, **kw)
        torch.cuda.synchronize()
        return cache.cpu(), None if scales is None else scales.cpu()

    def expected(self, skip=()):
        cache = self.cache.clone()
        scales = None if self.scales is None else self.scales.clone()
        for b, keep in enumerate(self.keep):
            for k, src in enumerate(keep):
                if (b, k) in skip:
                    continue
                dst = self.start[b] + k
                ps, pd = (int(self.table[b, p // self.bs]) for p in (src, dst))
                cache[pd, :, :, dst % self.bs] = cache[ps, :, :, src % self.bs]
                if scales is not None:
                    scales[pd, :, :, dst % self.bs] = scales[ps, :, :, src % self.bs]
        return cache, scales

    def check(self, skip=(), error=0):
        (c, s), (rc, rs) = self.run(), self.expected(skip)
        bits = (lambda t: t if t.dtype == torch.uint8 else t.view(torch.int16))
        assert torch.equal(bits(c), bits(rc))
        assert s is None or torch.equal(s, rs)
        assert pkv.get_device_error() == error


def subset(n, lo, hi, seed):
    g = torch.Generator().manual_seed(seed)
    return sorted((torch.randperm(hi - lo, generator=g)[:n] + lo).tolist())


@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (256, False), (64, True), (128, True)])
@pytest.mark.parametrize("bs", [8, 16, 128, 512])
def test_accepted_paths(d, fp8, bs):
    keep = [[100, 102, 103, 107], [50], [], list(range(7, 30)), [0, 1, 2]]
    c = Case(keep, [100, 43, 5, 7, 0], [120, 60, 20, 40, 3], d=d, fp8=fp8, bs=bs, seed=d + bs)
    c.check()


@pytest.mark.parametrize("hkv,batch", [(1, 1), (3, 1), (8, 2), (32, 40)])
def test_long_overlapping_moves(hkv, batch):
    """Sources and destinations overlap by every distance, chunk after chunk."""
    keep, start, lens = [], [], []
    for b in range(batch):
        n = 900 - 7 * b
        at = 3 + b
        k = subset(n, at + 1, at + 1 + int(n * (1.01 + 0.3 * (b % 3))) + 2, b)
        keep.append(k), start.append(at), lens.append(k[-1] + 1)
    c = Case(keep, start, lens, hkv=hkv, seed=hkv)
    c.check()


@pytest.mark.parametrize("shift", [1, 2, 15, 64, 65, 255, 256, 257, 1024])
def test_shift_by(shift):
    n = 2500
    for d, fp8 in ((64, True), (128, False), (256, False)):
        c = Case([list(range(shift + 4, shift + 4 + n))], [4], [n + shift + 4], hkv=1, d=d, fp8=fp8, seed=shift)
        c.check()


def test_any_order_and_repeats():
    """Only src >= dst is asked for: lists out of order, and one source listed more than once."""
    g = torch.Generator().manual_seed(1)
    keep = [int(k + torch.randint(0, 300, (1,), generator=g)) for k in range(1500)]
    c = Case([keep, [9, 9, 9, 5 + 3, 9]], [0, 5], [1900, 10], seed=2)
    c.check()


def test_more_rows_than_ctas():
    batch = 700
    keep = [[5 + (b % 3), 9, 11] for b in range(batch)]
    c = Case(keep, [4] * batch, [12] * batch, hkv=8, d=64, bs=8, seed=3)
    c.check()


def test_rows_out_of_range_are_skipped_and_flagged():
    keep = [[10, 4, 30, 12], [6, 7]]
    c = Case(keep, [8, 2], [32, 9], seed=4)
    c.check(skip={(0, 1)}, error=5)                      # behind its destination
    c = Case([[10, 10 ** 9, 15, 31], [6, 7]], [8, 2], [32, 9], seed=4)
    c.check(skip={(0, 1)}, error=5)                      # beyond the table
    c = Case([[10, 11, 30]], [8], [32], seed=5)
    c.table[0, 1] = -1                                   # position 30's page
    c.check(skip={(0, 2)}, error=5)
    c = Case([[10, 11, 30]], [8], [32], seed=5)
    c.table[0, 1] = 10 ** 6
    c.check(skip={(0, 2)}, error=5)
    c = Case([[10, 11], [20]], [-3, 18], [32, 32], seed=6)
    c.check(skip={(0, 0), (0, 1)}, error=5)              # a negative destination
    # cu_keep out of range: the sequence is skipped
    c = Case([[10, 11], [20]], [8, 18], [32, 32], seed=7)
    cache = c.cache.cuda()
    keep_pos, cu, start, table = c.args()
    cu[2] = 9
    pkv.kv_cache_compact(cache, keep_pos, cu, start, table)
    assert pkv.get_device_error() == 5
    assert torch.equal(cache.cpu().view(torch.int16), c.expected(skip={(1, 0)})[0].view(torch.int16))


def test_stream_and_graph():
    c = Case([[20, 22, 25], [8, 9]], [18, 3], [32, 16], seed=8)
    want, _ = c.expected()
    s = torch.cuda.Stream()
    got, _ = c.run(stream=s)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    cache, args = c.cache.cuda(), c.args()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_cache_compact(cache, *args)
    torch.cuda.synchronize()
    cache.copy_(c.cache)
    d = Case([[19, 30, 31], [5, 15]], [18, 3], [32, 16], seed=8)
    args[0].copy_(d.args()[0])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache.cpu().view(torch.int16), d.expected()[0].view(torch.int16))
