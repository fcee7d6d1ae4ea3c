"""How decodes are cut (csrc/decode_rules.h), compiled for the host: over an INT8 cache never more splits than over the others,
so that one workspace size serves every format; splits that the kernels can take; sizes before a device is usable."""
from __future__ import annotations

import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

import paged_kv_flash_cache_gb300 as pkv

HEADER = os.path.join(os.path.dirname(pkv.__file__), "csrc", "decode_rules.h")
SHIM = """
#include "%s"
extern "C" int split(int sms, int b, int hkv, int bs, int mb, int n) { return pkv::decode_split_tokens(sms, b, hkv, bs, mb, n); }
extern "C" void plan(int sms, int b, int hq, int hkv, int bs, int mb, int n, int *o) {
    const pkv::Int8Decode d = pkv::decode_int8_plan(sms, b, hq, hkv, bs, mb, n);
    o[0] = d.unit_heads; o[1] = d.cluster; o[2] = d.chunk; o[3] = d.wide;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("rules")
    (at / "shim.cpp").write_text(SHIM % HEADER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", str(at / "shim.so"), str(at / "shim.cpp")], check=True)
    return ctypes.CDLL(str(at / "shim.so"))


def plan(rules, *args):
    o = (ctypes.c_int * 4)()
    rules.plan(*args, o)
    return list(o)


def sizes(n):
    rng = random.Random(7)
    yield from [(3, 32, 32, 256, 39), (227, 32, 8, 64, 9), (11, 32, 32, 16, 192), (16, 32, 32, 16, 513), (1, 32, 8, 16, 2000),
                (64, 128, 1, 16, 513), (2500, 1, 1, 8, 5), (1, 1, 1, 512, 1 << 21)]
    for _ in range(n):
        heads = rng.choice([1, 2, 3, 4, 8, 16, 32])
        group = rng.choice([1, 2, 3, 4, 5, 8, 13, 16, 32, 64, 130])
        bs = rng.choice([8, 16, 32, 64, 128, 256, 512])
        yield int(2 ** rng.uniform(0, 11.5)), heads * group, heads, bs, max(1, int(2 ** rng.uniform(5, 18) / bs))


@pytest.mark.parametrize("sms", [152, 148, 20, 160])
def test_never_more_splits_than_the_other_formats(rules, sms):
    for batch, hq, heads, bs, mb in sizes(20000):
        cap = bs * mb
        for n in (0, 3):
            unit, cluster, chunk, wide = plan(rules, sms, batch, hq, heads, bs, mb, n)
            other = rules.split(sms, batch, heads, bs, mb, n)
            assert -(-cap // chunk) <= -(-cap // other), (batch, hq, heads, bs, mb, n)
            assert chunk % 128 == 0 and other % 128 == 0 and -(-cap // chunk) <= 2048
            group = hq // heads
            assert group % unit == 0 and unit <= (128 if wide else 8)
            assert wide == (cluster == 0 and group > 8)
            if cluster:
                assert n == 0 and batch * (hq // unit) * cluster <= (1 if cluster == 16 else 2) * sms


def test_fewer_sms_never_need_more(rules):
    """What is sized for 160 SMs holds for any number below."""
    for batch, hq, heads, bs, mb in sizes(5000):
        most = -(-bs * mb // rules.split(160, batch, heads, bs, mb, 0))
        for sms in (1, 60, 132, 148, 152):
            assert -(-bs * mb // rules.split(sms, batch, heads, bs, mb, 0)) <= most


def test_sizes_without_a_device(rules):
    if torch.cuda.is_available():
        pytest.skip("the sizes before a device is usable")
    lib = pkv.load_library()
    for batch, hq, heads, bs, mb in sizes(2000):
        old = lib.pkv_decode_workspace_size(batch, hq, heads, 128, bs, mb, 0)
        assert lib.pkv_decode_int8_workspace_size(batch, hq, heads, 128, bs, mb, 0) == old
        _, cluster, chunk, _ = plan(rules, 152, batch, hq, heads, bs, mb, 0)
        for c in (rules.split(152, batch, heads, bs, mb, 0), chunk):
            splits = -(-bs * mb // c)
            assert splits <= 1 or old >= batch * hq * splits * 129 * 4 + 16
    assert lib.pkv_decode_int8_workspace_size(0, 8, 8, 128, 16, 64, 0) == 0
    assert lib.pkv_decode_int8_workspace_size(4, 8, 3, 128, 16, 64, 0) == 0
