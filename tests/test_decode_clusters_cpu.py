"""The decode over an INT8 cache takes clusters of the sizes that the device can place, and splits where there are none."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from tests.test_decode_rules_cpu import HEADER, sizes

SHIM = """
#include "%s"
extern "C" void plan(int sms, int b, int hq, int hkv, int bs, int mb, int n, int clusters, int *o) {
    const pkv::Int8Decode d = pkv::decode_int8_plan(sms, b, hq, hkv, bs, mb, n, clusters);
    o[0] = d.unit_heads; o[1] = d.cluster; o[2] = d.chunk; o[3] = d.wide;
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("clusters")
    (at / "shim.cpp").write_text(SHIM % HEADER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-o", str(at / "shim.so"), str(at / "shim.cpp")], check=True)
    return ctypes.CDLL(str(at / "shim.so"))


def plan(rules, *args):
    o = (ctypes.c_int * 4)()
    rules.plan(*args, o)
    return list(o)


def test_clusters_that_the_device_can_place(rules):
    seen = set()
    for placeable in (31, 15, 7, 3, 1, 0, 5, 16):
        for batch, hq, heads, bs, mb in sizes(4000):
            unit, cluster, chunk, wide = plan(rules, 152, batch, hq, heads, bs, mb, 0, placeable)
            assert cluster == 0 or cluster & placeable == cluster
            assert chunk >= 128 and wide == (cluster == 0 and hq // heads > 8)
            seen.add((placeable, cluster))
    assert {(31, c) for c in (0, 1, 2, 4, 8, 16)} <= seen and {c for p, c in seen if p == 0} == {0}


def test_one_request_without_large_clusters(rules):
    # one request of 4096 tokens, 8 KV heads: clusters of 16; of 8 where those have no place, splits where a run would be long
    assert plan(rules, 152, 1, 32, 8, 16, 257, 0, 31)[1] == 16
    assert plan(rules, 152, 1, 32, 8, 16, 257, 0, 15)[1] == 8
    assert plan(rules, 152, 1, 32, 8, 16, 500, 0, 15)[1] == 0
