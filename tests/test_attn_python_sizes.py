"""Sizes that ctypes would cut to their low bits are refused by the Python calls of include/nmattn.h (CPU only)."""
import pytest
import torch

import sparse_matrix_vector_amd as nm


@pytest.mark.parametrize("sizes", ((4, 16 - 2 ** 32, 2, 64), (4 - 2 ** 64, 16, 2, 64), (4, 16, 2 - 2 ** 32, 64), (4, 16, 2, 64 - 2 ** 32)))
def test_caches(sizes):
    with pytest.raises(ValueError, match="no cache"):
        nm.KVCache(*sizes, torch.float16, device="cpu")


@pytest.mark.parametrize("B,hq,max_len,prefix_len", ((1 + 2 ** 64, 8, 100, 0), (1, 8 + 2 ** 32, 100, 0), (1, 8 - 2 ** 32, 100, 0),
                                                     (1, 8, 5000 + 2 ** 64, 0), (1, 8, 100 - 2 ** 64, 0), (1, 8, 100, 2 ** 64 + 1),
                                                     (1, 8, 100, 1 - 2 ** 64), (-1, 8, 100, 0)))
def test_workspaces(B, hq, max_len, prefix_len):
    cache = nm.KVCache(4, 16, 2, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="no such attention"):
        nm.attn_workspace(B, hq, cache, max_len, prefix_len)
    assert nm.attn_workspace(1, 8, cache, 5000, 100).numel() > 0


def test_frequencies():
    """2^31 + 32 frequencies are no rotation of 64 columns.  (The library is not called: no such tensor is made.)"""
    from sparse_matrix_vector_amd import attention as A
    assert A._rot(32) == 64 and A._rot(0) == 0
    for pairs in (2 ** 31 + 32, 2 ** 31 + 2 ** 30, 2 ** 62 + 8):
        assert not 0 <= A._rot(pairs) <= 512
