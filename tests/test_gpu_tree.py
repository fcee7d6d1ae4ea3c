"""paged_attn_tree on the GPU against attention computed in 64 bits from its definition: drafted nodes see the
context before them and the nodes of their mask row."""
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


class Case:
    """Random inputs: lens and nodes per sequence, mask rows (bool [nodes, nodes] a sequence) and the paged cache."""

    def __init__(self, lens, nodes, hq, hkv, d=128, bs=16, dtype="bf16", seed=0, masks="tree", spare=2, max_q=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.nodes, self.hq, self.hkv, self.d, self.bs, self.dt = lens, nodes, hq, hkv, d, bs, DT[dtype]
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + spare
        order = torch.randperm(nb, generator=g).tolist()
        mb = max(max(need), 1) + 1
        self.table = torch.full((len(lens), mb), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
            at += k
        self.cache = torch.randn((nb, 2, hkv, bs, d), generator=g).to(self.dt)
        self.q = torch.randn((sum(nodes), hq, d), generator=g).to(self.dt)
        self.max_q = max(nodes + [1]) if max_q is None else max_q
        words = (self.max_q + 31) // 32
        self.sees = []
        rows = []
        for b, n in enumerate(nodes):
            if masks == "tree":
                par = [-1 if i == 0 else int(torch.randint(-1, i, (1,), generator=g)) for i in range(n)]
                m = W.tree_mask([par], self.max_q)
            else:  # any set
                m = torch.randint(-2 ** 31, 2 ** 31, (n, words), generator=g, dtype=torch.int64).to(torch.int32)
            rows.append(m)
            bits = ((m[:, :, None].long() >> torch.arange(32)) & 1).bool().flatten(1)
            self.sees.append(bits[:, :n].clone())
        self.mask = torch.cat(rows) if rows else torch.zeros((0, words), dtype=torch.int32)
        self.cu = W.cu_lens(nodes)

    def hide(self, b, i, j):
        """Node i of sequence b does not see node j."""
        r, w = int(self.cu[b]) + i, j // 32
        v = int(self.mask[r, w]) & 0xFFFFFFFF & ~(1 << (j % 32))
        self.mask[r, w] = v - (1 << 32) if v >= 1 << 31 else v
        self.sees[b][i, j] = False

    def slot(self, b, pos):
        return int(self.table[b, pos // self.bs]), pos % self.bs

    def run(self, **kw):
        dev = {k: getattr(self, k).cuda() for k in ("cache", "q", "mask", "cu", "table")}
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        out = pkv.paged_attn_tree(dev["cache"], dev["q"], dev["mask"], dev["cu"], lens, dev["table"],
                                  max_q_len=self.max_q, lse=lse, **kw)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def exact(self, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        outs, lses, vmax, smax = [], [], 0.0, 0.0
        for b, (n, L) in enumerate(zip(self.nodes, self.lens)):
            pages = self.table[b, :-(-L // self.bs)].long()
            kv = self.cache[pages].double().permute(1, 2, 0, 3, 4).reshape(2, self.hkv, -1, self.d)[:, :, :L]
            vis = torch.cat([torch.ones((n, L - n), dtype=torch.bool), self.sees[b]], 1)
            q = self.q[int(self.cu[b]):int(self.cu[b + 1])].double()
            for i in range(n):
                k, v = kv[0][:, vis[i]], kv[1][:, vis[i]]          # only what the node sees
                s = torch.einsum("hgd,hpd->hgp", q[i].reshape(self.hkv, -1, self.d), k) * scale
                if s.shape[-1] == 0:
                    outs.append(torch.zeros((self.hq, self.d), dtype=torch.float64))
                    lses.append(torch.full((self.hq,), -math.inf, dtype=torch.float64))
                    continue
                smax = max(smax, float((q[i].abs().sum(-1).max() * k.abs().max()).nan_to_num(0, 0, 0)) * scale)
                lse = torch.logsumexp(s, -1)
                o = torch.einsum("hgp,hpd->hgd", torch.exp(s - lse[..., None]), v)
                outs.append(o.reshape(self.hq, self.d))
                lses.append(lse.reshape(self.hq))
                vmax = max(vmax, float(v.abs().masked_fill(~v.isfinite(), 0).max()))
        return torch.stack(outs), torch.stack(lses), vmax

    def p_half(self, dtype):
        """Half a step of the 16-bit type where P is rounded to it: 16-bit outputs, head_dim up to 128 and blocks of more than
        128 rows (nodes x heads of a unit); otherwise P has two parts."""
        unit = self.hq // self.hkv
        unit = next(u for u in range(min(unit, 128), 0, -1) if unit % u == 0)
        wide = self.d <= 128 and self.max_q > 128 // unit and dtype != torch.float32
        return torch.finfo(dtype).eps / 2 if wide else 0.0

    def check(self, got, what="", scale=None):
        """Tolerances. A score is a sum of D products of 16-bit values in FP32: off by at most D * 2^-24 of the sum of their
        magnitudes, here (N(0, 1) rows, scale D^-1/2) below D * 2^-24 * 0.9 * D^1/2; ex2 and the two-part P add 2^-17
        relative; numerator and denominator: twice that. So an output is within 2 (0.9 D^3/2 2^-24 + 2^-17) max|v|, plus half
        a step of its type. Where P is rounded to 16 bits (p_half), each weight is off by half a step of itself: half a step of
        max|v| more."""
        (out, lse), (ro, rl, vmax) = got, self.exact(scale)
        rel = 0.9 * self.d ** 1.5 * 2.0 ** -24
        tol = 2 * (rel + 2.0 ** -17) * vmax + self.p_half(out.dtype) * vmax
        half = torch.finfo(out.dtype).eps / 2
        fin = ro.isfinite()
        assert torch.equal(out.double().isfinite(), fin), what
        err = (out.double() - ro).abs()[fin]
        assert (err <= tol + half * 1.01 * ro.abs()[fin] + 1e-7).all(), (what, float(err.max()), tol)
        assert torch.equal(lse == -math.inf, rl == -math.inf), what
        f = rl.isfinite()
        assert ((lse.double() - rl).abs()[f] <= rel + 2.0 ** -20 * (1 + rl.abs()[f])).all(), what
        assert pkv.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,bs", [(64, 8), (128, 16), (256, 32), (128, 128), (64, 512)])
def test_one_small_tree(d, bs, dtype):
    c = Case([100], [9], 8, 2, d=d, bs=bs, dtype=dtype, seed=d + bs)
    c.check(c.run())


# group 1, 2, 4 ... with one tile, two tiles (129 rows and more at head_dim up to 128), several row blocks
@pytest.mark.parametrize("hq,hkv,n", [(4, 4, 1), (4, 4, 128), (4, 4, 129), (4, 4, 300), (8, 2, 32), (8, 2, 33),
                                      (8, 2, 64), (8, 2, 65), (6, 2, 43), (32, 1, 4), (32, 1, 5), (32, 1, 17),
                                      (128, 1, 1), (128, 1, 3), (131, 1, 2), (160, 1, 3), (40, 4, 31)])
def test_groups_and_row_blocks(hq, hkv, n):
    c = Case([n + 333, n, n + 5], [n, n, max(1, n // 2)], hq, hkv, seed=hq + n)
    c.check(c.run(), (hq, hkv, n))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_ragged_batch(d):
    lens = [1, 2, 127, 128, 129, 1, 700, 1500, 64, 257, 300, 2047]
    nodes = [1, 2, 3, 64, 65, 0, 31, 17, 64, 1, 40, 63]
    c = Case(lens, nodes, 8, 2, d=d, bs=16, seed=d)
    c.check(c.run())


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 90, (400,), generator=g).tolist()
    nodes = [int(torch.randint(0, min(20, L) + 1, (1,), generator=g)) for L in lens]
    c = Case(lens, nodes, 2, 1, d=64, bs=8, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 200])
def test_any_mask(n):
    c = Case([n + 100, n], [n, n], 4, 2, d=64, seed=n, masks="any")
    c.check(c.run(), n)


@pytest.mark.parametrize("ctx", [0, 1, 96, 97, 127, 128, 129, 255])
def test_tree_across_tile_borders(ctx):
    c = Case([ctx + 70], [70], 8, 4, seed=ctx)
    c.check(c.run(), ctx)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_context_is_split(d):
    # one item split over many runs; several splits meeting inside one run
    c = Case([20011], [7], 4, 1, d=d, bs=64, seed=1)
    c.check(c.run())
    c = Case([9000, 5000, 12000], [40, 64, 3], 8, 2, d=d, bs=32, seed=2)
    c.check(c.run())


def test_rows_that_see_nothing():
    for d in (64, 128, 256):
        c = Case([20, 300], [20, 9], 8, 2, d=d, seed=5)
        for j in range(20):
            c.hide(0, 7, j)
            c.hide(0, 19, j)
        out, lse = c.run()
        c.check((out, lse))
        assert (out[7] == 0).all() and (lse[7] == -math.inf).all() and (lse[19] == -math.inf).all()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d,hq", [(64, 4), (128, 4), (128, 16), (256, 4)])
def test_what_is_masked_may_hold_anything(bad, d, hq):
    """Infinities and NaN in K and V: of nodes that only some see, of rows behind the context, of pages not
    listed; the nodes that do see them get what the definition gives."""
    n = 40
    c = Case([150, n], [n, n], hq, 2, d=d, seed=9, masks="any")
    for b, L in enumerate(c.lens):
        for i in range(n):
            for j in (3, 38):
                if i != j and i % 3:
                    c.hide(b, i, j)
        for pos in range(L, -(-L // c.bs) * c.bs):   # behind the context, in its last page
            p, o = c.slot(b, pos)
            c.cache[p, :, :, o] = bad
        p, o = c.slot(b, L - n + 3)
        c.cache[p, 1, :, o] = bad                    # V of node 3: a whole row
        p, o = c.slot(b, L - n + 38)
        c.cache[p, 1, 0, o, 5] = bad                 # V of node 38: one element of one head
    used = set(c.table[c.table >= 0].tolist())
    for p in set(range(c.cache.shape[0])) - used:
        c.cache[p] = bad
    out, lse = c.run()
    c.check((out, lse))
    ro, _, _ = c.exact()
    assert torch.equal(out.isnan(), ro.isnan())
    inf = ro.isinf()
    assert torch.equal(out[inf].double(), ro[inf])
    # K of a node that nobody else sees
    c = Case([150], [n], hq, 2, d=d, seed=10)
    for i in range(n):
        c.hide(0, i, 11)
    p, o = c.slot(0, 150 - n + 11)
    c.cache[p, :, :, o] = bad
    c.check(c.run())


def test_scale_and_fp32_output():
    c = Case([400], [33], 8, 2, seed=11)
    out, lse = c.run(scale=0.03, out_dtype=torch.float32)
    assert out.dtype == torch.float32
    c.check((out, lse), scale=0.03)


def test_large_scores():
    # scores of +-200: the running max jumps and rows settle on single keys
    c = Case([600], [20], 4, 2, seed=12)
    c.q *= 16
    out, lse = c.run()
    ro, rl, vmax = c.exact()
    # scores 16 times as large, so are their errors (see Case.check)
    tol = 2 * (16 * 0.9 * 128 ** 1.5 * 2.0 ** -24 + 2.0 ** -17) * vmax
    assert ((out.double() - ro).abs() <= tol + 2.0 ** -8 * ro.abs()).all()
    assert ((lse.double() - rl).abs() <= 16 * 0.9 * 128 ** 1.5 * 2.0 ** -24 + 2.0 ** -20 * rl.abs()).all()


def test_rows_behind_the_last_sequence_are_left():
    c = Case([100, 60], [5, 9], 4, 2, seed=13)
    pad = 6
    q = torch.cat([c.q, torch.full((pad, 4, 128), math.nan, dtype=c.dt)]).cuda()
    mask = torch.cat([c.mask, torch.full((pad, c.mask.shape[1]), -1, dtype=torch.int32)]).cuda()
    out = torch.full(q.shape, 3.0, dtype=c.dt, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    pkv.paged_attn_tree(c.cache.cuda(), q, mask, c.cu.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(),
                        c.table.cuda(), max_q_len=9, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[-pad:] == 3.0).all() and (lse[-pad:] == 3.0).all()
    c.check((out[:-pad].cpu(), lse[:-pad].cpu()))


def test_lengths_out_of_range_are_skipped_and_flagged():
    c = Case([100, 60, 200], [5, 9, 4], 4, 2, seed=14)
    good, _ = c.run()
    dev = [t.cuda() for t in (c.cache, c.q, c.mask, c.cu, c.table)]
    cap = c.table.shape[1] * c.bs
    for lens, max_q, cu in (([100, 8, 200], 9, None), ([100, cap + 1, 200], 9, None), ([100, -1, 200], 9, None),
                            ([100, 60, 200], 8, None)):
        out = torch.full(c.q.shape, 3.0, dtype=c.dt, device="cuda")
        pkv.paged_attn_tree(dev[0], dev[1], dev[2], dev[3], torch.tensor(lens, dtype=torch.int32).cuda(), dev[4],
                            max_q_len=max_q, out=out)
        assert pkv.get_device_error() == 5
        out = out.cpu()
        assert (out[5:14] == 3.0).all()
        assert torch.equal(out[:5], good[:5]) and torch.equal(out[14:], good[14:])
    # rows beyond q
    out = torch.full(c.q.shape, 3.0, dtype=c.dt, device="cuda")
    cu = torch.tensor([0, 5, 14, 19], dtype=torch.int32).cuda()
    pkv.paged_attn_tree(dev[0], dev[1], dev[2], cu, torch.tensor(c.lens, dtype=torch.int32).cuda(), dev[4],
                        max_q_len=9, out=out)
    assert pkv.get_device_error() == 5
    assert (out[14:] == 3.0).all() and torch.equal(out[:14].cpu(), good[:14])


def test_bad_page_is_flagged_and_page_zero_read():
    c = Case([100], [5], 4, 2, seed=15)
    c.table[0, 2] = 10 ** 6
    c.run()
    assert pkv.get_device_error() == 5
    c.table[0, 2] = 0
    c.check(c.run())


def test_workspace_contents_do_not_matter_and_calls_repeat():
    c = Case([3000, 900], [40, 64], 8, 2, seed=16)
    need = pkv.tree_workspace_size(8, 2, 128, 64)
    a = c.run(workspace=torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda"))
    b = c.run(workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(a)


def test_streams_and_graphs():
    c = Case([2500, 130], [30, 12], 8, 2, seed=17)
    want, _ = c.run()
    cache, q, mask, cu, table = (t.cuda() for t in (c.cache, c.q, c.mask, c.cu, c.table))
    lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    ws = [torch.empty(pkv.tree_workspace_size(8, 2, 128, 30), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):  # two calls at once, a workspace each
        for s, w, o in zip(side, ws, outs):
            pkv.paged_attn_tree(cache, q, mask, cu, lens, table, max_q_len=30, workspace=w, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_attn_tree(cache, q, mask, cu, lens, table, max_q_len=30, workspace=ws[0], out=outs[0])
    for k in (1, 2, 3):  # new queries, lengths and masks in the captured tensors
        d = Case([2500 - 300 * k, 130 - k], [30 - k, 12], 8, 2, seed=17 + k, max_q=30)
        d.cache, d.table = c.cache, c.table
        rows = int(d.cu[-1])
        q[:rows].copy_(d.q)
        mask[:rows].copy_(d.mask)
        cu.copy_(d.cu)
        lens.copy_(torch.tensor(d.lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ro, _, vmax = d.exact()
        tol = 2 * (0.9 * 128 ** 1.5 * 2.0 ** -24 + 2.0 ** -17) * vmax
        assert ((outs[0][:rows].cpu().double() - ro).abs() <= tol + 1.01 * 2.0 ** -8 * ro.abs()).all()


def test_a_chain_is_causal_prefill():
    """A chain of drafted tokens is the causal chunk that paged_attn_prefill attends."""
    n = 24
    c = Case([500, n + 7], [n, n], 8, 2, seed=18)
    chain = W.tree_mask([list(range(-1, n - 1))] * 2)
    c.mask = chain
    c.sees = [torch.ones((n, n), dtype=torch.bool).tril()] * 2
    c.check(c.run())
    out, _ = c.run(out_dtype=torch.float32)
    ref = pkv.paged_attn_prefill(c.cache.cuda(), c.q.cuda(), c.cu.cuda(), torch.tensor(c.lens, dtype=torch.int32).cuda(),
                                 c.table.cuda(), max_q_len=n, out_dtype=torch.float32)
    # the prefill rounds P to 16 bits: half a step of each weight, so 2^-8 max|v| on both sides of the quotient
    assert (out - ref.cpu()).abs().max() <= 2.0 ** -8 * float(c.cache.float().abs().max())
