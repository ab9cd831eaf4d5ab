"""Workspaces of the serving operators' calls: what one call needs, and what serves every smaller one (CPU: sizes are host
code); on the GPU, that a call without a workspace takes what it needs and no more."""
import ctypes
import random

import pytest
import torch

import sparse_matrix_vector_amd as nm
from sparse_matrix_vector_amd import _lib as L

BF16 = torch.bfloat16


def sizes(op):
    lib = L.serve_lib()
    return getattr(lib, f"nm_attn_{op}_call_bytes"), getattr(lib, f"nm_attn_{op}_workspace_bytes")


def test_plans_of_one_range_need_nothing():
    call, _ = sizes("tree")
    for args in ((256, 24, 64, 8, 128, 1, 4096), (256, 24, 64, 8, 128, 1, 512), (64, 24, 32, 8, 128, 1, 4096),
                 (1, 8, 32, 8, 128, 0, 300), (4, 64, 8, 8, 64, 1, 0)):
        assert call(*args) == 0, args
    call, _ = sizes("prompt")
    for args in ((8192, 8192, 1, 64, 8, 128), (1024, 1024, 1, 32, 8, 256), (5000, 5000, 16, 32, 8, 128), (0, 0, 0, 1, 1, 64)):
        assert call(*args) == 0, args


def test_bad_sizes():
    call, _ = sizes("prompt")
    for bad in ((-1, 1, 1, 8, 8, 64), (1, 2 ** 31 - 2 ** 16, 1, 8, 8, 64), (1, 1, 65536, 8, 8, 64), (1, 1, 1, 7, 2, 64),
                (1, 1, 1, 8, 8, 80), (1, 1, 65535, 65535, 65535, 64), (2 ** 27, 1, 1, 65528, 8, 64)):
        assert call(*bad) == -1
    call, _ = sizes("tree")
    for bad in ((0, 1, 8, 8, 64, 0, 1), (1, 0, 8, 8, 64, 0, 1), (1, 65, 8, 8, 64, 0, 1), (1, 1, 7, 2, 64, 0, 1),
                (1, 1, 8, 8, 80, 0, 1), (1, 1, 8, 8, 64, 3, 1), (1, 1, 8, 8, 64, 0, -1), (1, 1, 8, 8, 64, 0, 2 ** 31),
                (65535, 64, 17, 17, 64, 0, 1)):
        assert call(*bad) == -1


def test_a_byte_less_is_refused():
    """The calls ask for just what the *_call_bytes functions say (addresses are never followed: the calls are refused)."""
    a = [0x100000000 * (i + 1) for i in range(8)]
    lib = L.serve_lib()
    need = lib.nm_attn_prompt_call_bytes(16, 20000, 1, 4, 2, 128)
    assert need > 0
    for ws, nb in ((None, 0), (None, need), (a[6], need - 1)):
        assert lib.nm_attn_prompt(a[0], 512, 16, a[1], 256, a[2], 256, 20000, a[3], a[4], 1, 4, 2, 128, 1, 0.1, a[5], None, ws,
                                  nb, None) == L.NM_ERR_INVALID_ARG
    c = L.KvCacheStruct(k=a[0], v=a[1], k_scale=None, v_scale=None, n_pages=4, page_size=16, heads=2, D=64, dtype=1, format=0)
    need = lib.nm_attn_tree_call_bytes(3, 8, 4, 2, 64, 0, 100000)
    assert need > 0
    assert lib.nm_attn_tree(a[2], 256, 3, 8, 4, ctypes.byref(c), a[3], a[4], 6250, a[5], 100000, 0.1, a[6], None, a[7],
                            need - 1, None) == L.NM_ERR_INVALID_ARG


def test_one_calls_need_is_within_every_larger_bound():
    r = random.Random(5)
    call, bound = sizes("tree")
    for _ in range(3000):
        heads, G, D, fmt = r.choice((1, 2, 8, 16)), r.choice((1, 3, 4, 8)), r.choice((64, 128, 256)), r.randint(0, 2)
        N, B, ml = r.randint(1, 64), r.randint(1, 300), int(2 ** r.uniform(0, 18))
        most = bound(B, N, heads * G, heads, D, fmt, ml)
        for b, m in ((B, ml), (r.randint(1, B), ml), (B, r.randint(0, ml)), (r.randint(1, B), r.randint(0, ml))):
            assert 0 <= call(b, N, heads * G, heads, D, fmt, m) <= most
    call, bound = sizes("prompt")
    for _ in range(3000):
        heads, G, D = r.choice((1, 2, 8, 16)), r.choice((1, 3, 4, 8)), r.choice((64, 128, 256))
        T, Tk, B = int(2 ** r.uniform(0, 14)), int(2 ** r.uniform(0, 18)), r.randint(1, 64)
        most = bound(T, Tk, B, heads * G, heads, D)
        for t, tk, b in ((T, Tk, B), (r.randint(0, T), Tk, B), (T, r.randint(0, Tk), r.randint(0, B))):
            assert 0 <= call(t, tk, b, heads * G, heads, D) <= most


def test_tree_bound_is_near_some_calls_need():
    """A sequence that is not cut has no partial results.  Those that are make no more than 512 / u + B' ranges together (u
    units each, B' u < 512), and about 512 / u for some number of them: within a factor of three with the rounding of ranges."""
    call, bound = sizes("tree")
    for heads, G, N, D, fmt, B, ml in ((8, 8, 24, 128, 1, 256, 4096), (8, 4, 24, 128, 1, 64, 4096), (8, 4, 12, 128, 0, 32, 2048),
                                       (8, 8, 24, 128, 1, 256, 200), (16, 8, 64, 128, 2, 500, 4096), (64, 1, 64, 64, 0, 500, 1000),
                                       (8, 4, 12, 128, 0, 100, 16384)):
        args = lambda b, m: (b, N, heads * G, heads, D, fmt, m)                                             # noqa: E731
        largest = max(call(*args(b, m)) for b in range(1, B + 1) for m in {ml, ml // 2 + 1, min(ml, 512), min(ml, 513)})
        assert largest <= bound(*args(B, ml)) <= 3 * largest, (heads, G, N, B, ml)


# ---- on the GPU ------------------------------------------------------------------
def taken(f):
    """Most bytes that f() holds of the allocator beyond what is there."""
    f()                                                 # whatever is made once
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    f()
    return torch.cuda.max_memory_allocated() - before


def near(got, need):
    return need <= got < need + 512 if need else got == 0       # the allocator's blocks are of 512 bytes


@pytest.mark.gpu
def test_prompt_takes_what_it_needs():
    for T, Tk, B, hq, heads, D in ((700, 700, 1, 8, 2, 128), (512, 512, 1, 4, 1, 256), (16, 9000, 1, 8, 2, 128)):
        q = torch.zeros((T, hq, D), dtype=BF16, device="cuda")
        k = torch.zeros((Tk, heads, D), dtype=BF16, device="cuda")
        st, kst = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (T, Tk))
        out = torch.empty_like(q)
        need = sizes("prompt")[0](T, Tk, B, hq, heads, D)
        assert (need > 0) == (T == 16)
        assert near(taken(lambda: nm.attn_prompt(q, k, k, st, kst, out=out)), need)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert taken(lambda: nm.attn_prompt(q, k, k, st, kst, out=out, ws=ws)) == 0


@pytest.mark.gpu
def test_tree_takes_what_it_needs():
    for B, N, hq, heads, ml in ((64, 24, 32, 8, 512), (128, 8, 32, 8, 1024), (1, 8, 8, 2, 300), (2, 24, 32, 8, 4096)):
        cache = nm.KVCache(4, 64, heads, 128, BF16, "mx8")
        q = torch.zeros((B, N, hq, 128), dtype=BF16, device="cuda")
        table = torch.zeros((B, ml // 64 + 1), dtype=torch.int32, device="cuda")
        lens = torch.full((B,), 64, dtype=torch.int32, device="cuda")
        visible = torch.zeros((B, N), dtype=torch.int64, device="cuda")
        out = torch.empty_like(q)
        need = sizes("tree")[0](B, N, hq, heads, 128, 1, ml)
        assert (need > 0) == (B == 2)
        assert near(taken(lambda: nm.attn_tree(q, cache, table, lens, visible, max_len=ml, out=out)), need)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        assert taken(lambda: nm.attn_tree(q, cache, table, lens, visible, max_len=ml, out=out, ws=ws)) == 0
