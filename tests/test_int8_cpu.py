"""INT8 caches and page calls without a GPU: what the calls refuse, and the reference of the append against the bounds
that the format promises."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv
from tests import int8_ref


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


def _cache(ptr=4096, nb=4, hkv=2, bs=16, d=128, dt=0, fmt=2, scales=4096):
    return pkv._Cache(ptr, nb, hkv, bs, d, dt, fmt, scales)


P, F, good = ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p(4096)


def test_int8_cache_refusals(lib):
    app = lambda c, n=0: lib.pkv_kv_cache_append(c, good, good, good, good, good, 1, 4, n, None)
    assert app(_cache()) == 0
    assert app(_cache(scales=None)) == 1
    assert app(_cache(scales=4100)) == 1
    assert app(_cache(ptr=4104)) == 1
    assert app(_cache(d=256)) == 2
    assert app(_cache(d=96)) == 2
    assert app(_cache(bs=24)) == 2
    assert app(_cache(dt=2)) == 2
    assert lib.pkv_kv_cache_append(_cache(), P(4104), good, good, good, good, 1, 4, 3, None) == 1
    assert lib.pkv_kv_cache_append(_cache(), good, good, None, good, good, 1, 4, 3, None) == 1
    # calls that place rows one by one, or move them between pages
    rope = pkv._Rope(0, 0, None, 1.0, None, None, 1e-6)
    assert lib.pkv_rope_append(_cache(), rope, good, 256, 2, good, 256, good, 256, good, good, good, good, 1, 4, 3,
                               good, 256, None) == 2
    assert lib.pkv_paged_attn_tree(_cache(), good, 2, good, 1, good, good, good, 1, 4, 4, 4, F(0.1), good, 1 << 30, good,
                                   0, None, None) == 2
    assert lib.pkv_kv_cache_compact(_cache(), good, good, good, good, 1, 4, 3, None) == 2


def test_page_call_refusals(lib):
    copy = lambda d, s, n=0, a=good, b=good: lib.pkv_kv_cache_copy(d, s, a, b, None, n, None)
    for fmt, scales in ((0, None), (1, 4096), (2, 4096)):
        c = _cache(fmt=fmt, scales=scales)
        assert copy(c, c) == 0
        assert copy(c, c, n=-1) == 1
        assert copy(c, c, n=3, a=None) == 1
        assert copy(c, c, n=3, b=None) == 1
    assert copy(_cache(), _cache(fmt=1)) == 1
    assert copy(_cache(), _cache(d=64)) == 1
    assert copy(_cache(), _cache(bs=32)) == 1
    assert copy(_cache(), _cache(hkv=4)) == 1
    assert copy(_cache(fmt=0, scales=None), _cache(fmt=0, scales=None, dt=1)) == 1
    assert copy(_cache(ptr=None), _cache()) == 1
    assert copy(_cache(), _cache(), n=1) in (0, 4) if not torch.cuda.is_available() else True

    def fork(n=2, m=2, mb=4, tables=P(8192), lens=P(12288), parents=P(16384), fresh=P(20480), out=P(24576), out_lens=P(28672)):
        return lib.pkv_kv_cache_fork(_cache(), tables, lens, parents, fresh, n, m, mb, out, out_lens, None)
    assert fork(m=0) == 0
    assert fork(n=-1) == 1 and fork(m=-1) == 1 and fork(mb=0) == 1
    assert fork(tables=None) == 1 and fork(parents=None) == 1 and fork(out=None) == 1
    # outputs over inputs: in place, by a part, lengths over tables
    assert fork(out=P(8192)) == 1
    assert fork(out=P(8192 + 16)) == 1
    assert fork(out_lens=P(8192 + 28)) == 1
    assert fork(out_lens=P(12288)) == 1
    assert fork(out=P(28672)) == 1
    assert fork(out=P(16384)) == 1 and fork(out_lens=P(20480)) == 1


def test_binding_refuses_int8_caches_without_their_scales():
    cache = torch.zeros((4, 2, 2, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        pkv._cache_struct(cache, torch.float16, None)
    with pytest.raises(ValueError):
        pkv._cache_struct(cache, torch.float16, torch.zeros((4, 2, 2, 16)))
    with pytest.raises(ValueError):
        pkv._cache_struct(cache, torch.float16, torch.zeros((4, 2, 2), dtype=torch.float64))


def test_least_power_of_two():
    for a in (127.0, 127.00001, 1.0, 126.9, 2.0 ** -119, 3e38, 1e-40, 0.9921875, 0.99218756):
        s = int8_ref.least_power_of_two(a)
        assert a <= 127 * s and s >= 2.0 ** -126
        assert s == 2.0 ** -126 or a > 127 * s / 2


@pytest.mark.parametrize("bs", [8, 64])
def test_a_value_is_off_by_less_than_a_step_however_often_its_scale_grew(bs):
    # rows of growing magnitude, one a call: the scale of the page grows nearly every time
    rng = np.random.default_rng(bs)
    k = rng.standard_normal((bs, 2, 64)) * (1.9 ** (np.arange(bs) % 16))[:, None, None]
    v = rng.standard_normal((bs, 2, 64)) * (1.3 ** np.arange(bs))[:, None, None]
    codes, scales = np.zeros((1, 2, 2, bs, 64), np.int8), np.zeros((1, 2, 2), np.float32)
    tables = np.zeros((1, 1), np.int32)
    for t in range(bs):
        int8_ref.append(codes, scales, k[t:t + 1], v[t:t + 1], [0, 1], [t], tables)
    kv = int8_ref.context(codes, scales, tables[0], bs)
    for i, x in enumerate((k, v)):
        err = np.abs(kv[i] - x.transpose(1, 0, 2))
        assert np.all(err < scales[0, i].astype(np.float64)[:, None, None])
        # the last rows were written with the last scale: half a step
        assert np.all(err[:, -1] <= scales[0, i].astype(np.float64)[:, None] / 2)


def test_one_call_or_several():
    """A page that one call fills holds each value to half a step; the scale is the same either way."""
    rng = np.random.default_rng(5)
    k, v = rng.standard_normal((2, 40, 3, 64))
    tables = np.array([[2, 0, 1]], np.int32)
    one, s1 = np.zeros((3, 2, 3, 16, 64), np.int8), np.zeros((3, 2, 3), np.float32)
    many, s2 = one.copy(), s1.copy()
    int8_ref.append(one, s1, k, v, [0, 40], [0], tables)
    at = 0
    for n in (1, 7, 16, 2, 14):
        int8_ref.append(many, s2, k[at:at + n], v[at:at + n], [0, n], [at], tables)
        at += n
    assert at == 40 and np.array_equal(s1, s2)
    kv = int8_ref.context(one, s1, tables[0], 40)
    step = np.repeat(s1[[2, 0, 1]].transpose(1, 2, 0), 16, 2)[:, :, :40, None]
    assert np.all(np.abs(kv - np.stack((k, v)).transpose(0, 2, 1, 3)) <= step / 2)
    assert np.all(np.abs(int8_ref.context(many, s2, tables[0], 40) - kv) <= 1.0 * step)
