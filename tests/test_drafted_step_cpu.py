"""Refusals of rope_append, paged_attn_tree and kv_cache_compact before anything is launched, and their host-side
helpers: no GPU needed."""
import ctypes
import math

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import build as pkv_build
from paged_kv_flash_cache_gb300 import rope
from paged_kv_flash_cache_gb300 import workloads as W

P, F = ctypes.c_void_p, ctypes.c_float
GOOD = P(4096)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load_library()


def cache(ptr=4096, nb=4, hkv=2, bs=16, d=128, dt=0, fmt=0, scales=None):
    return pkv._Cache(P(ptr), nb, hkv, bs, d, dt, fmt, None if scales is None else P(scales))


def call_rope(lib, c=None, **kw):
    a = dict(rot=128, inter=0, inv=GOOD, mscale=1.0, qw=None, kw=None, eps=1e-6, q=GOOD, qs=512, hq=4, k=GOOD, ks=256,
             v=GOOD, vs=256, pos=GOOD, cu=GOOD, before=GOOD, bt=GOOD, batch=1, mb=4, n=3, out=GOOD, os=512)
    a.update(kw)
    r = pkv._Rope(a["rot"], a["inter"], a["inv"], a["mscale"], a["qw"], a["kw"], a["eps"])
    return lib.pkv_rope_append(c or cache(), r, a["q"], a["qs"], a["hq"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["cu"],
                               a["before"], a["bt"], a["batch"], a["mb"], a["n"], a["out"], a["os"], None)


def test_rope_append_refusals(lib):
    for kw in (dict(rot=-16), dict(rot=144), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(mscale=math.nan),
               dict(mscale=math.inf), dict(qs=511), dict(qs=516), dict(ks=248), dict(ks=260), dict(vs=128), dict(os=504),
               dict(hq=0), dict(batch=-1), dict(n=-1), dict(mb=0), dict(inv=None), dict(q=None), dict(k=None), dict(v=None),
               dict(pos=None), dict(cu=None), dict(before=None), dict(bt=None), dict(out=None), dict(q=P(4100)),
               dict(k=P(4104)), dict(v=P(4098)), dict(out=P(4100)), dict(qw=P(4100)), dict(kw=P(4104))):
        assert call_rope(lib, **kw) == INVALID, kw
    assert call_rope(lib, out=P(8192), q=P(8192), os=520) == INVALID   # in place: q's own stride
    assert call_rope(lib, rot=24) == UNSUPPORTED
    assert call_rope(lib, cache(d=96)) == UNSUPPORTED
    assert call_rope(lib, cache(ptr=0)) == INVALID
    assert call_rope(lib, cache(d=256, fmt=1, scales=4096), ks=512, vs=512, qs=1024, os=1024) == UNSUPPORTED
    assert call_rope(lib, batch=0) == 0 and call_rope(lib, n=0) == 0


def call_tree(lib, c=None, **kw):
    a = dict(q=GOOD, hq=4, mask=GOOD, words=1, cu=GOOD, lens=GOOD, bt=GOOD, batch=1, mb=4, total=8, most=8, scale=0.1,
             ws=GOOD, bytes=1 << 40, out=GOOD, dt=0, lse=None)
    a.update(kw)
    return lib.pkv_paged_attn_tree(c or cache(), a["q"], a["hq"], a["mask"], a["words"], a["cu"], a["lens"], a["bt"],
                                   a["batch"], a["mb"], a["total"], a["most"], F(a["scale"]), a["ws"], a["bytes"], a["out"],
                                   a["dt"], a["lse"], None)


def test_tree_refusals(lib):
    for kw in (dict(hq=3), dict(hq=0), dict(batch=-1), dict(mb=0), dict(total=-1), dict(most=-1), dict(words=-1),
               dict(words=0), dict(most=33), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
               dict(q=None), dict(mask=None), dict(cu=None), dict(lens=None), dict(bt=None), dict(out=None), dict(q=P(4100)),
               dict(out=P(4104)), dict(lse=P(4100))):
        assert call_tree(lib, **kw) == INVALID, kw
    assert call_tree(lib, dt=1) == UNSUPPORTED          # bf16 out of an fp16 cache
    assert call_tree(lib, mb=1 << 27) == UNSUPPORTED    # 2^31 tokens
    assert call_tree(lib, cache(d=256, fmt=1, scales=4096)) == UNSUPPORTED
    assert call_tree(lib, cache(fmt=1)) == INVALID      # an FP8 cache without its scales
    assert call_tree(lib, cache(d=96)) == UNSUPPORTED
    need = pkv.tree_workspace_size(4, 2, 128, 8)
    assert call_tree(lib, bytes=need - 1) == WORKSPACE
    assert call_tree(lib, ws=None) == WORKSPACE
    assert call_tree(lib, ws=P(4104)) == WORKSPACE
    for kw in (dict(batch=0), dict(total=0), dict(most=0)):
        assert call_tree(lib, **kw) == 0


def test_tree_workspace_size(lib):
    # 160 runs: a 32-byte item and two partials of 128 rows (one tile) or 256 (two) of D outputs and an lse
    def size(rows, d):
        return 160 * (32 + 2 * rows * (d + 1) * 4)
    assert pkv.tree_workspace_size(32, 8, 128, 32) == size(128, 128)   # 32 nodes x 4 heads: one tile
    assert pkv.tree_workspace_size(32, 8, 128, 33) == size(256, 128)
    assert pkv.tree_workspace_size(32, 8, 256, 33) == size(128, 256)   # head_dim 256: tiles one by one
    assert pkv.tree_workspace_size(32, 8, 64, 1000) == size(256, 64)
    assert pkv.tree_workspace_size(3, 2, 128, 8) == 0
    assert pkv.tree_workspace_size(4, 2, 128, 0) == 0


def test_compact_refusals(lib):
    def call(c=None, keep=GOOD, cu=GOOD, to=GOOD, bt=GOOD, batch=2, mb=4, n=5):
        return lib.pkv_kv_cache_compact(c or cache(), keep, cu, to, bt, batch, mb, n, None)
    for kw in (dict(keep=None), dict(cu=None), dict(to=None), dict(bt=None), dict(batch=-1), dict(mb=0), dict(n=-1)):
        assert call(**kw) == INVALID, kw
    assert call(cache(bs=24)) == UNSUPPORTED
    assert call(cache(fmt=1)) == INVALID
    assert call(cache(nb=1 << 26, hkv=2, bs=16)) == UNSUPPORTED    # 2^32 rows
    assert call(cache(nb=1 << 30, hkv=1 << 30, bs=512)) == UNSUPPORTED
    assert call(batch=0) == 0 and call(n=0) == 0


def test_tree_mask_and_depths():
    par = [[-1, 0, 0, 1, 3, -1], [], [-1]]
    m = W.tree_mask(par)
    assert m.shape == (7, 1) and m.dtype == torch.int32
    assert [int(x) for x in m[:, 0]] == [0b1, 0b11, 0b101, 0b1011, 0b11011, 0b100000, 0b1]
    assert W.tree_depths(par).tolist() == [0, 1, 1, 2, 3, 0, 0]
    chain = W.tree_mask([list(range(-1, 69))], max_q_len=100)
    assert chain.shape == (70, 4)
    assert [x & 0xFFFFFFFF for x in chain[69].tolist()] == [0xFFFFFFFF, 0xFFFFFFFF, 0x3F, 0]
    for bad in ([[0]], [[-1, 2, 0]], [[-2]]):
        with pytest.raises(ValueError):
            W.tree_mask(bad)


def test_rope_frequencies():
    f, m = rope.rope_frequencies(64, 10000.0)
    assert f.dtype == torch.float32 and f.shape == (32,) and m == 1.0
    assert float(f[0]) == 1.0 and float(f[16]) == pytest.approx(0.01, rel=1e-6)
    lin, _ = rope.rope_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin, f / 4, rtol=1e-6)
    ntk, _ = rope.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert float(ntk[0]) == 1.0 and float(ntk[-1]) == pytest.approx(float(f[-1]) / 4, rel=1e-5)
    for kind in ("parts", "smooth"):
        g, m = rope.rope_frequencies(128, 10000.0, scaling=kind, factor=8.0, original_length=4096)
        h, _ = rope.rope_frequencies(128, 10000.0)
        ratio = (g / h).double()
        assert float(ratio[0]) == 1.0 and float(ratio[-1]) == pytest.approx(1 / 8, rel=1e-6)
        assert (ratio.diff() <= 1e-6).all()
        assert m == (pytest.approx(0.1 * math.log(8) + 1) if kind == "parts" else 1.0)
        turns = 4096 * h.double() / (2 * math.pi)
        # pairs well above the fast end are kept, pairs below the slow end divided by the factor
        fast = 32.0 if kind == "parts" else 4.0
        assert (ratio[turns > fast * 1.2] == 1.0).all()
        assert ((ratio[turns < 0.8] - 1 / 8).abs() < 1e-6).all()
    one, m = rope.rope_frequencies(64, scaling="parts", factor=1.0, original_length=100)
    assert torch.equal(one, f) and m == 1.0
    for kw in (dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=64, scaling="other"),
               dict(rotary_dim=64, scaling="parts", factor=2.0), dict(rotary_dim=64, factor=0.5),
               dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, scaling="smooth", original_length=10, fast=1.0)):
        with pytest.raises(ValueError):
            rope.rope_frequencies(**kw)


def test_bindings_refuse_what_does_not_fit():
    """Shape and device checks that need no GPU: CPU tensors are refused, there is no CPU path."""
    c = torch.zeros((4, 2, 2, 16, 64), dtype=torch.float16)
    bt = torch.zeros((1, 4), dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((3, 4, 64), dtype=torch.float16)
    k = torch.zeros((3, 2, 64), dtype=torch.float16)
    for call in (lambda: pkv.kv_cache_compact(c, one, one, one[:1], bt),
                 lambda: pkv.paged_attn_tree(c, q, torch.zeros((3, 1), dtype=torch.int32), one, one[:1], bt, max_q_len=3),
                 lambda: pkv.rope_append(c, q, k, k, torch.ones(32), one, one[:1], bt,
                                         positions=torch.zeros(3, dtype=torch.int32))):
        with pytest.raises((ValueError, RuntimeError)):
            call()
