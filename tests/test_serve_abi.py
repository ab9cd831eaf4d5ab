"""CPU checks of include/nmserve.h: every declared call is exported and bound,
sizes and refusals (argument checks are host code; nothing here reaches the
GPU), and the Python layer's own checks."""
import ctypes
import math
import os
import re

import pytest
import torch

import sparse_matrix_vector_amd as nm
from sparse_matrix_vector_amd import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nmserve.h")

# Distinct, 256-byte aligned addresses that are never followed.
ADDR = [0x100000000 * (i + 1) for i in range(16)]


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(nm_\w+)\s*\(", text, flags=re.M)))


def test_header_library_and_binding_agree():
    lib = L.serve_lib()
    assert declared() == sorted(L.SERVE_SIGNATURES)
    for name in declared():
        assert hasattr(lib, name)
    text = re.search(r"typedef struct \{(.*?)\} nm_kv_pages;", open(HEADER).read(), flags=re.S).group(1)
    assert re.findall(r"(\w+);", text) == [name for name, _ in L.KvPagesStruct._fields_]


def test_every_call_is_public():
    for name in ("KVPages", "kv_plan", "attn_prompt", "attn_prompt_workspace", "attn_tree", "attn_tree_workspace"):
        assert name in nm.__all__ and getattr(nm, name).__doc__


# ---- the book of pages ---------------------------------------------------------
def plan(pages=True, adds=ADDR[5], rows=64, starts=ADDR[6], slots=ADDR[7], positions=ADDR[8], granted=ADDR[9], **kw):
    d = dict(table=ADDR[0], lens=ADDR[1], free=ADDR[2], n_free=ADDR[3], scratch=ADDR[4], B=8, width=16, n_pages=100, page_size=64)
    d.update(kw)
    return L.serve_lib().nm_kv_plan(ctypes.byref(L.KvPagesStruct(**d)) if pages else None, adds, rows, starts, slots,
                                    positions, granted, None)


@pytest.mark.parametrize("kw,want", [
    (dict(pages=False), 1), (dict(B=0), 2), (dict(B=65536), 2), (dict(B=-1), 2), (dict(width=0), 2),
    (dict(width=2 ** 24 + 1), 2), (dict(B=128, width=2 ** 24), 2), (dict(n_pages=0), 2), (dict(n_pages=2 ** 31), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2), (dict(page_size=-16), 2), (dict(rows=-1), 2),
    (dict(rows=2 ** 31), 2), (dict(rows=2 ** 31 - 1, slots=None), 1),
    *((dict([(name, None)]), 1) for name in ("table", "lens", "free", "n_free", "scratch", "adds", "starts", "slots", "positions",
                                             "granted")),
    *((dict([(name, ADDR[15] + 2)]), 1) for name in ("table", "lens", "free", "n_free", "adds", "starts", "positions", "granted")),
    (dict(scratch=ADDR[4] + 4), 1), (dict(slots=ADDR[7] + 4), 1),
    (dict(table=ADDR[5]), 1), (dict(granted=ADDR[5]), 1), (dict(lens=ADDR[5] + 28), 1), (dict(free=ADDR[0] + 8 * 16 * 4 - 4), 1),
    (dict(n_free=ADDR[2] + 396), 1), (dict(scratch=ADDR[1]), 1), (dict(starts=ADDR[9] - 32), 1), (dict(slots=ADDR[8] - 8), 1),
    (dict(positions=ADDR[7] + 508), 1)])
def test_plan_refusals(kw, want):
    assert plan(**kw) == want


def test_plan_scratch():
    f = L.serve_lib().nm_kv_plan_scratch_bytes
    assert f(0) == f(-1) == f(65536) == f(2 ** 40) == -1
    sizes = [f(B) for B in range(1, 2000)]
    assert all(4 * (B + 1) <= n and n % 8 == 0 for B, n in zip(range(1, 2000), sizes)) and sizes == sorted(sizes)


# ---- prompts -------------------------------------------------------------------
def prompt(q=ADDR[0], qs=512, T=100, k=ADDR[1], ks=256, v=ADDR[2], vs=256, Tk=200, starts=ADDR[3], k_starts=ADDR[4], B=2, Hq=4,
           heads=2, D=128, dt=1, scale=0.1, o=ADDR[5], lse=None, ws=ADDR[6], nb=1 << 28):
    return L.serve_lib().nm_attn_prompt(q, qs, T, k, ks, v, vs, Tk, starts, k_starts, B, Hq, heads, D, dt, scale, o, lse, ws,
                                        nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), 3), (dict(dt=-1), 3), (dict(T=-1), 2), (dict(T=2 ** 31), 2), (dict(Tk=-1), 2), (dict(Tk=2 ** 31 - 2 ** 16), 2),
    (dict(B=-1), 2), (dict(B=65536), 2), (dict(B=65535, Hq=16385, heads=16385, qs=16385 * 128, ks=16385 * 128, vs=16385 * 128), 2),
    (dict(Hq=0), 2), (dict(Hq=5), 2), (dict(heads=0), 2), (dict(Hq=65536), 2), (dict(D=96), 2), (dict(D=512), 2),
    (dict(T=2 ** 30 - 2 ** 15), 2), (dict(k_starts=None), 2), (dict(qs=504), 2), (dict(qs=516), 2), (dict(ks=248), 2),
    (dict(vs=260), 2), (dict(ks=2 ** 28 + 8), 2), (dict(qs=2 ** 28 + 8), 2), (dict(scale=math.nan), 2), (dict(scale=-math.inf), 2),
    (dict(scale=1.1e30), 2), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(starts=None), 1), (dict(o=None), 1),
    (dict(q=ADDR[0] + 8), 1), (dict(k=ADDR[1] + 2), 1), (dict(v=ADDR[2] + 4), 1), (dict(starts=ADDR[3] + 2), 1),
    (dict(k_starts=ADDR[4] + 1), 1), (dict(o=ADDR[5] + 8), 1), (dict(lse=ADDR[7] + 2), 1), (dict(ws=ADDR[6] + 16), 1),
    (dict(nb=-1), 1), (dict(o=ADDR[0]), 1), (dict(o=ADDR[1] + 16), 1), (dict(o=ADDR[4] - 16), 1), (dict(lse=ADDR[5] + 64), 1),
    (dict(lse=ADDR[3] + 8), 1), (dict(ws=ADDR[5]), 1), (dict(ws=ADDR[2]), 1),
    (dict(T=16, Tk=20000, B=1, ws=None), 1), (dict(T=16, Tk=20000, B=1, nb=1024), 1)])
def test_prompt_refusals(kw, want):
    assert prompt(**kw) == want


def test_empty_prompts():
    assert prompt(T=0, q=None, o=None) == 0 and prompt(B=0, Tk=100, starts=None, k_starts=None) == 0
    assert prompt(T=0, Tk=0, q=None, k=None, v=None, o=None, k_starts=None) == 0
    assert prompt(T=0, Tk=0, B=0, q=None, k=None, v=None, o=None, starts=None, k_starts=None, ws=None, nb=0) == 0


def test_prompt_workspace_bytes():
    f = L.serve_lib().nm_attn_prompt_workspace_bytes
    assert f(16, 20000, 1, 32, 8, 128) > 0 and f(8192, 100, 1, 32, 8, 128) == 0 and f(0, 0, 0, 1, 1, 64) == 0
    for bad in ((-1, 1, 1, 8, 8, 64), (1, 2 ** 31 - 2 ** 16, 1, 8, 8, 64), (1, 1, 65536, 8, 8, 64), (1, 1, 1, 7, 2, 64),
                (1, 1, 1, 8, 8, 80), (1, 1, 65535, 65535, 65535, 64), (2 ** 27, 1, 1, 65528, 8, 64)):
        assert f(*bad) == -1


# ---- trees ---------------------------------------------------------------------
def cache(**kw):
    d = dict(k=ADDR[8], v=ADDR[9], k_scale=ADDR[10], v_scale=ADDR[11], n_pages=4, page_size=16, heads=2, D=128, dtype=1,
             format=1)
    d.update(kw)
    return L.KvCacheStruct(**d)


def tree(c, q=ADDR[0], qs=512, B=3, N=8, Hq=4, visible=ADDR[5], table=ADDR[1], stride=4, lens=ADDR[2], ml=64, scale=0.1, o=ADDR[3],
         lse=None, ws=ADDR[4], nb=1 << 24):
    return L.serve_lib().nm_attn_tree(q, qs, B, N, Hq, ctypes.byref(c) if c else None, visible, table, stride, lens, ml, scale,
                                      o, lse, ws, nb, None)


@pytest.mark.parametrize("kw,want", [(dict(dtype=2), 3), (dict(format=3), 3), (dict(format=-1), 3), (dict(n_pages=0), 2),
                                     (dict(page_size=24), 2), (dict(heads=0), 2), (dict(D=96), 2), (dict(k=None), 1),
                                     (dict(v_scale=None), 1), (dict(k=ADDR[8] + 8), 1)])
def test_tree_bad_caches(kw, want):
    assert tree(cache(**kw)) == want
    assert tree(None) == L.NM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 2), (dict(B=65536), 2), (dict(N=0), 2), (dict(N=65), 2), (dict(N=-1), 2), (dict(Hq=0), 2), (dict(Hq=5), 2),
    (dict(B=65535, N=64, Hq=18, qs=2304), 2), (dict(ml=-1), 2), (dict(ml=2 ** 30 + 1), 2), (dict(qs=504), 2), (dict(qs=516), 2),
    (dict(scale=math.nan), 2), (dict(scale=math.inf), 2), (dict(scale=-1.1e30), 2), (dict(stride=3), 2),
    (dict(q=None), 1), (dict(o=None), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(visible=None), 1),
    (dict(visible=ADDR[5] + 4), 1), (dict(q=ADDR[0] + 2), 1), (dict(o=ADDR[3] + 8), 1), (dict(lens=ADDR[2] + 2), 1),
    (dict(ws=ADDR[4] + 16), 1), (dict(o=ADDR[0]), 1), (dict(o=ADDR[5] - 16), 1), (dict(lse=ADDR[3] + 64), 1), (dict(o=ADDR[8]), 1),
    (dict(ws=ADDR[10]), 1), (dict(lse=ADDR[2]), 1), (dict(nb=-1), 1), (dict(ws=ADDR[3]), 1),
    (dict(ml=100000, stride=6250, ws=None), 1), (dict(ml=100000, stride=6250, nb=1024), 1)])
def test_tree_refusals(kw, want):
    assert tree(cache(), **kw) == want


def test_tree_workspace_bytes():
    f = L.serve_lib().nm_attn_tree_workspace_bytes
    assert f(1, 4, 32, 8, 128, 0, 100) == 0 and f(4, 64, 8, 8, 64, 1, 0) == 0
    assert f(32, 12, 64, 8, 128, 2, 4096) > 0
    for bad in ((0, 1, 8, 8, 64, 0, 1), (1, 0, 8, 8, 64, 0, 1), (1, 65, 8, 8, 64, 0, 1), (1, 1, 7, 2, 64, 0, 1),
                (1, 1, 8, 8, 80, 0, 1), (1, 1, 8, 8, 64, 3, 1), (1, 1, 8, 8, 64, 0, -1), (1, 1, 8, 8, 64, 0, 2 ** 31),
                (65535, 64, 17, 17, 64, 0, 1)):
        assert f(*bad) == -1


# ---- the Python layer ----------------------------------------------------------
def test_python_refuses_host_tensors():
    x, i = torch.zeros((2, 2, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    book, c = nm.KVPages(2, 4, 8, 16, device="cpu"), nm.KVCache(4, 16, 2, 64, torch.float16, device="cpu")
    masks = torch.zeros((1, 2), dtype=torch.int64)
    for f in (lambda: nm.kv_plan(book, i, 4), lambda: nm.attn_prompt(x, x, x, i),
              lambda: nm.attn_tree(x.view(1, 2, 2, 64), c, i.view(1, 2), i[:1], masks)):
        with pytest.raises(TypeError, match="CUDA"):
            f()
    with pytest.raises(TypeError, match="KVPages"):
        nm.kv_plan(c, i, 4)
    with pytest.raises(TypeError, match="KVCache"):
        nm.attn_tree(x.view(1, 2, 2, 64), book, i.view(1, 2), i[:1], masks)


def test_new_books():
    book = nm.KVPages(3, 5, 7, 32, device="cpu")
    assert book.lens.tolist() == [0] * 3 and book.n_free.tolist() == [7] and book.free.tolist() == [6, 5, 4, 3, 2, 1, 0]
    assert book.table.shape == (3, 5) and (book.sequences, book.width, book.n_pages, book.page_size) == (3, 5, 7, 32)
    with pytest.raises(AttributeError):
        book.table = book.lens


@pytest.mark.parametrize("sizes", [(0, 4, 8, 16), (65536, 4, 8, 16), (2, 0, 8, 16), (2, 2 ** 24 + 1, 8, 16), (128, 2 ** 24, 8, 16),
                                   (2, 4, 0, 16), (2, 4, 8, 24), (2, 4, 8, 512), (2 + 2 ** 64, 4, 8, 16), (2, 4 - 2 ** 64, 8, 16),
                                   (2, 4, 8, 16 + 2 ** 32), (2, 4, 8 + 2 ** 64, 16)])
def test_no_such_book(sizes):
    with pytest.raises(ValueError, match="no book"):
        nm.KVPages(*sizes, device="cpu")


@pytest.mark.parametrize("sizes", [(16 + 2 ** 64, 20000, 1, 32, 8, 128), (16, 20000 - 2 ** 64, 1, 32, 8, 128), (16, 20000, 1 + 2 ** 64, 32, 8, 128),
                                   (16, 20000, 1, 32 + 2 ** 32, 8, 128), (16, 20000, 1, 32, 8 + 2 ** 32, 128),
                                   (16, 20000, 1, 32, 8, 128 - 2 ** 32), (-1, 20000, 1, 32, 8, 128), (16, 20000, 1, 33, 8, 128)])
def test_no_such_prompt_workspace(sizes):
    with pytest.raises(ValueError, match="no such attention"):
        nm.attn_prompt_workspace(*sizes, device="cpu")
    assert nm.attn_prompt_workspace(16, 20000, 1, 32, 8, 128, device="cpu").numel() > 0


@pytest.mark.parametrize("B,N,hq,ml", [(1 + 2 ** 64, 8, 8, 100), (1, 8 + 2 ** 32, 8, 100), (1, 8, 8 - 2 ** 32, 100), (1, 8, 8, 100 + 2 ** 64),
                                       (1, 65, 8, 100), (0, 8, 8, 100)])
def test_no_such_tree_workspace(B, N, hq, ml):
    c = nm.KVCache(4, 16, 2, 64, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="no such attention"):
        nm.attn_tree_workspace(B, N, hq, c, ml)
    assert nm.attn_tree_workspace(4, 8, 8, c, 5000).numel() > 0
