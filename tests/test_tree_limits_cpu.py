"""Sizes that paged_attn_tree does not take, on the host: no GPU needed."""
import pytest

import paged_kv_flash_cache_gb300 as pkv
from paged_kv_flash_cache_gb300 import workloads as W
from tests.test_drafted_step_cpu import UNSUPPORTED, cache, call_tree, lib  # noqa: F401


@pytest.mark.parametrize("head_dim", [8, 32, 80, 96, 192, 512, 1 << 30])
def test_no_workspace_for_head_dims_that_are_refused(lib, head_dim):  # noqa: F811
    assert pkv.tree_workspace_size(4, 2, head_dim, 8) == 0
    assert call_tree(lib, cache(d=head_dim)) == UNSUPPORTED


@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_workspace_for_those_that_are_not(lib, head_dim):  # noqa: F811
    assert pkv.tree_workspace_size(4, 2, head_dim, 8) == 160 * (32 + 2 * 128 * (head_dim + 1) * 4)


def test_pools_of_2_31_rows_are_refused(lib):  # noqa: F811
    """The rows of the pool are TMA coordinates of 32 bits with a sign. (An FP8 pool of so many rows of 64 bytes has 137 GB.)"""
    for c in (cache(nb=1 << 22, hkv=32, bs=8), cache(nb=1 << 21, hkv=8, bs=64, d=64, fmt=1, scales=4096),
              cache(nb=(1 << 31) - 1, hkv=1 << 30, bs=512)):
        assert call_tree(lib, c, hq=c.num_kv_heads) == UNSUPPORTED
    # one page less: refused for something else (a workspace of one byte), or not at all
    for c in (cache(nb=(1 << 22) - 1, hkv=32, bs=8), cache(nb=(1 << 21) - 1, hkv=8, bs=64, d=64, fmt=1, scales=4096)):
        assert call_tree(lib, c, hq=c.num_kv_heads, bytes=1) == 3


@pytest.mark.parametrize("parents", [[[0]], [[-1, 2, 0]], [[-2]], [[-1], [-1, 0, -3]]])
def test_depths_refuse_the_parents_that_masks_refuse(parents):
    for make in (W.tree_mask, W.tree_depths):
        with pytest.raises(ValueError):
            make(parents)
