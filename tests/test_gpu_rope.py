"""rope_append on the GPU against norm, rotation and placement computed in 64 bits."""
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import rope
from paged_kv_flash_cache_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_flash_cache_gb300 import build
    build.build()
    assert torch.cuda.is_available()


class Case:
    def __init__(self, new, before, hq, hkv, d=128, rot=None, bs=16, dtype="bf16", seed=0, inter=False, norm=False,
                 mscale=1.0, fp8=False, fused=True, far=0, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.before, self.hq, self.hkv, self.d, self.bs = new, before, hq, hkv, d, bs
        self.dt, self.inter, self.mscale, self.fp8, self.eps = DT[dtype], inter, mscale, fp8, 1e-5
        self.rot = d if rot is None else rot
        need = [max(1, -(-(b + n) // bs)) for n, b in zip(new, before)]
        nb = sum(need) + 2
        order = torch.randperm(nb, generator=g).tolist()
        self.table = torch.full((len(new), max(need) + 1), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
            at += k
        shape = (nb, 2, hkv, bs, d)
        if fp8:
            self.cache = torch.randint(0, 120, shape, generator=g, dtype=torch.uint8)
            self.scales = torch.rand(shape[:4], generator=g)
        else:
            self.cache, self.scales = torch.randn(shape, generator=g).to(self.dt), None
        total = sum(new) + pad
        self.total = sum(new)
        x = torch.randn((total, (hq + 2 * hkv) * d), generator=g).to(self.dt)
        self.x = x
        self.fused = fused
        self.positions = torch.cat([torch.arange(n) + b for n, b in zip(new, before)] + [torch.zeros(pad)]).to(torch.int32) + far
        self.inv_freq, _ = rope.rope_frequencies(self.rot) if self.rot else (torch.empty(0), 1.0)
        self.qw = self.kw = None
        if norm:
            self.qw, self.kw = (1 + 0.2 * torch.randn((2, d), generator=g)).to(self.dt).unbind(0)

    def views(self, x):
        hq, hkv, d = self.hq, self.hkv, self.d
        q, k, v = x.split([hq * d, hkv * d, hkv * d], 1)
        out = [q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))]
        return out if self.fused else [t.contiguous() for t in out]

    def run(self, **kw):
        q, k, v = self.views(self.x.cuda())
        cache = self.cache.cuda()
        scales = None if self.scales is None else self.scales.cuda()
        w = [None if t is None else t.cuda() for t in (self.qw, self.kw)]
        out = pkv.rope_append(cache, q, k, v, self.inv_freq.cuda(), W.cu_lens(self.new).cuda(),
                              torch.tensor(self.before, dtype=torch.int32).cuda(), self.table.cuda(),
                              positions=self.positions.cuda(), interleaved=self.inter, mscale=self.mscale,
                              q_weight=w[0], k_weight=w[1], eps=self.eps, scales=scales, **kw)
        torch.cuda.synchronize()
        return out.cpu(), cache.cpu(), None if scales is None else scales.cpu()

    def turned(self, x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + self.eps) * w.double()
        if not self.rot:
            return x
        t = torch.outer(self.positions.double(), self.inv_freq.double())[:, None]
        c, s = t.cos() * self.mscale, t.sin() * self.mscale
        y = x.clone()
        i = torch.arange(self.rot // 2)
        a, b = (2 * i, 2 * i + 1) if self.inter else (i, i + self.rot // 2)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        return y

    def rows(self):
        """(page, offset) of every new token."""
        for b, (n, at) in enumerate(zip(self.new, self.before)):
            for i in range(n):
                yield int(self.table[b, (at + i) // self.bs]), (at + i) % self.bs

    def check(self, got):
        """Tolerances: the angle's fraction of a turn is off by at most 2^-24 (its product) + 2^-25 (to FP32), so the
        angle by 2 pi 2^-23; sine, cosine and the norm's rsqrt by a few 2^-24. With |(a, b)| the pair's length, a rotated
        element is within 2^-20 |(a, b)| before its rounding, which adds half a step."""
        out, cache, scales = got
        q, k, v = self.views(self.x)
        n = self.total
        rq, rk = self.turned(q, self.qw)[:n], self.turned(k, self.kw)[:n]

        def near(x, ref):
            half = torch.finfo(x.dtype).eps / 2
            tiny = torch.finfo(x.dtype).smallest_normal * half * 2
            length = ref.square().amax(-1, keepdim=True).sqrt() * 2 ** 0.5
            err = (x.double() - ref).abs()
            assert (err <= half * ref.abs() + 2.0 ** -20 * (1 + half) * length + tiny).all(), float(err.max())

        near(out[:n], rq)
        where = list(self.rows())
        page, off = (torch.tensor([w[i] for w in where], dtype=torch.long) for i in (0, 1))
        if not self.fp8:
            near(cache[page, 0, :, off], rk)
            assert torch.equal(cache[page, 1, :, off].view(torch.int16), v[:n].contiguous().view(torch.int16))
            rest = self.cache.clone()
            rest[page, :, :, off] = cache[page, :, :, off]
            assert torch.equal(rest.view(torch.int16), cache.view(torch.int16)), "something else was written"
        else:
            sk = rk.abs().amax(-1) / 448.0
            gk = scales[page, 0, :, off].double()
            assert ((gk - sk).abs() <= 2.0 ** -19 * sk).all()
            deq = cache[page, 0, :, off].view(torch.float8_e4m3fn).double() * gk[..., None]
            # half a step of e4m3 (2^-4 of the value, 2^-10 of a scale below its normal range), and the value's own error
            assert ((deq - rk).abs() <= rk.abs() * 2.0 ** -4 * 1.001 + sk[..., None] * (2.0 ** -10 + 448 * 2.0 ** -19)).all()
            rest, rs = self.cache.clone(), self.scales.clone()
            rest[page, :, :, off] = cache[page, :, :, off]
            rs[page, :, :, off] = scales[page, :, :, off]
            assert torch.equal(rest, cache) and torch.equal(rs, scales)
            # V as kv_cache_append writes it
            c2, s2 = self.cache.cuda(), self.scales.cuda()
            pkv.kv_cache_append(c2, k[:n].contiguous().cuda(), v[:n].contiguous().cuda(), W.cu_lens(self.new).cuda(),
                                torch.tensor(self.before, dtype=torch.int32).cuda(), self.table.cuda(), scales=s2)
            assert torch.equal(c2.cpu()[page, 1, :, off], cache[page, 1, :, off])
            assert torch.equal(s2.cpu()[page, 1, :, off], scales[page, 1, :, off])
        assert pkv.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 96), (128, 0), (256, 256), (256, 64),
                                   (256, 208)])
def test_layouts_and_partial_rotation(d, rot, inter, dtype):
    for norm in (False, True):
        c = Case([5, 17], [3, 30], 4, 2, d=d, rot=rot, dtype=dtype, inter=inter, norm=norm, seed=d + rot, mscale=1.1)
        c.check(c.run())


@pytest.mark.parametrize("hq,hkv", [(1, 1), (32, 32), (32, 8), (12, 3), (71, 1), (5, 5)])
@pytest.mark.parametrize("new", [[1], [1] * 40, [300, 1, 0, 77]])
def test_heads_and_lengths(hq, hkv, new):
    c = Case(new, [(7 * i) % 50 for i in range(len(new))], hq, hkv, seed=hq, norm=True)
    c.check(c.run())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_fp8_cache(d, inter):
    c = Case([9, 40, 1], [0, 21, 100], 8, 4, d=d, rot=d // 2, dtype="bf16", fp8=True, inter=inter, norm=True, seed=d)
    c.check(c.run())
    c = Case([33], [5], 6, 6, d=d, dtype="f16", fp8=True, inter=inter, seed=d + 1)
    c.check(c.run())


def test_fp8_zero_rows():
    c = Case([4], [0], 2, 2, fp8=True, seed=3)
    c.x[1] = 0
    out, cache, scales = c.run()
    p, o = list(c.rows())[1]
    assert (scales[p, :, :, o] == 0).all() and (cache[p, :, :, o] == 0).all()


@pytest.mark.parametrize("far", [0, 1, 131072, 10 ** 6, 2 ** 30, -5, 2 ** 31 - 10, -2 ** 31 + 10])
def test_far_positions(far):
    c = Case([6], [0], 4, 2, far=0, seed=1)
    c.positions = (torch.arange(6, dtype=torch.int64) + far).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32)
    c.check(c.run())


def test_frequencies_of_any_size():
    c = Case([6], [1000], 4, 2, seed=2)
    c.inv_freq = torch.logspace(-9, 3, 64, dtype=torch.float64).float()
    c.inv_freq[3] = 0.0
    c.inv_freq[5] = -0.7
    c.check(c.run())


def test_in_place_contiguous_and_spaced_tokens():
    for fused in (False, True):
        c = Case([20, 3], [2, 9], 8, 2, fused=fused, norm=True, seed=4)
        want, _, _ = c.run()
        x = c.x.cuda()
        q, k, v = c.views(x)
        cache = c.cache.cuda()
        got = pkv.rope_append(cache, q, k, v, c.inv_freq.cuda(), W.cu_lens(c.new).cuda(),
                              torch.tensor(c.before, dtype=torch.int32).cuda(), c.table.cuda(),
                              positions=c.positions.cuda(), q_weight=c.qw.cuda(), k_weight=c.kw.cuda(), eps=c.eps, q_out=q)
        torch.cuda.synchronize()
        assert got.data_ptr() == q.data_ptr() and torch.equal(q.cpu(), want)


def test_norm_of_one_side_only_and_large_values():
    c = Case([10], [0], 4, 2, norm=True, seed=5)
    c.kw = None
    c.check(c.run())
    c = Case([10], [0], 4, 2, norm=True, seed=5)
    c.x = (c.x.double() * 1e4).to(c.dt)
    c.qw = None
    c.check(c.run())


def test_padded_tokens_and_bad_slots():
    c = Case([5, 6], [0, 10], 4, 2, seed=6, pad=7)
    q_out = torch.full((18, 4, 128), 3.0, dtype=c.dt, device="cuda")
    got = c.run(q_out=q_out)
    c.check(got)
    assert (got[0][11:] == 3.0).all()
    # a page outside the pool, a position beyond the table, a negative one: skipped, the queries still written
    for table, before in (((1, 0, 9999), None), ((1, 0, -1), None), (None, 10 ** 6), (None, -20)):
        c = Case([5, 6], [0, 10], 4, 2, seed=6)
        want = c.run()
        if table:
            c.table[table[0], table[1]] = table[2]
        else:
            c.before = [0, before]
        out, cache, _ = c.run()
        assert pkv.get_device_error() == 5
        assert torch.equal(out, want[0])
        p, o = int(c.table[0, 0]), 0
        assert torch.equal(cache[p, :, :, :5], want[1][p, :, :, :5])


def test_streams_and_graph_replay():
    c = Case([1] * 8, [5 * i for i in range(8)], 8, 2, seed=7)
    want = c.run()
    x = c.x.cuda()
    q, k, v = c.views(x)
    cache, out = c.cache.cuda(), torch.empty((8, 8, 128), dtype=c.dt, device="cuda")
    args = (c.inv_freq.cuda(), W.cu_lens(c.new).cuda(), torch.tensor(c.before, dtype=torch.int32).cuda(), c.table.cuda())
    pos = c.positions.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.rope_append(cache, q, k, v, *args, positions=pos, q_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out.cpu(), want[0]) and torch.equal(cache.cpu(), want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rope_append(cache, q, k, v, *args, positions=pos, q_out=out)
    d = Case([1] * 8, [5 * i for i in range(8)], 8, 2, seed=8)
    d.table, d.cache = c.table, c.cache
    x.copy_(d.x)
    pos.copy_(d.positions)
    cache.copy_(c.cache)
    g.replay()
    torch.cuda.synchronize()
    d.check((out.cpu(), cache.cpu(), None))


def test_no_rotation_no_norm_is_the_append():
    c = Case([50, 3], [7, 0], 4, 2, rot=0, seed=9)
    out, cache, _ = c.run()
    q, k, v = c.views(c.x)
    ref = c.cache.cuda()
    pkv.kv_cache_append(ref, k.contiguous().cuda(), v.contiguous().cuda(), W.cu_lens(c.new).cuda(),
                        torch.tensor(c.before, dtype=torch.int32).cuda(), c.table.cuda())
    assert torch.equal(ref.cpu(), cache) and torch.equal(out, q)
