"""CPU checks of include/nmattn.h: every declared call is exported and bound,
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
HEADER = os.path.join(ROOT, "include", "nmattn.h")

# Distinct, 256-byte aligned addresses that are never followed.
ADDR = [0x100000000 * (i + 1) for i in range(16)]


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:int|int64_t)\s+(nm_\w+)\s*\(", text, flags=re.M)))


def test_header_library_and_binding_agree():
    lib = L.attn_lib()
    assert declared() == sorted(L.ATTN_SIGNATURES)
    for name in declared():
        assert hasattr(lib, name)


@pytest.mark.parametrize("args,want", [((10, 64, 8, 128, 0), 10 * 64 * 8 * 256), ((10, 64, 8, 128, 1), 10 * 64 * 8 * 128),
                                       ((3, 16, 1, 64, 2), 3 * 16 * 32), ((0, 64, 8, 128, 0), -1), ((1, 48, 8, 128, 0), -1),
                                       ((1, 8, 8, 128, 0), -1), ((1, 512, 8, 128, 0), -1), ((1, 64, 0, 128, 0), -1),
                                       ((1, 64, 8, 96, 0), -1), ((1, 64, 8, 128, 3), -1), ((1, 64, 8, 128, -1), -1),
                                       ((2 ** 31, 64, 8, 128, 0), -1), ((2 ** 31 - 1, 256, 65535, 256, 0), -1),
                                       ((-1, 64, 8, 128, 0), -1)])
def test_cache_bytes(args, want):
    assert L.attn_lib().nm_kv_bytes(*args) == want
    if want < 0:
        assert L.attn_lib().nm_kv_scale_bytes(*args) == -1


def test_cache_scale_bytes():
    lib = L.attn_lib()
    assert lib.nm_kv_scale_bytes(10, 64, 8, 128, 0) == 0
    assert lib.nm_kv_scale_bytes(10, 64, 8, 128, 1) == lib.nm_kv_scale_bytes(10, 64, 8, 128, 2) == 10 * 64 * 8 * 4


def qk(q=ADDR[0], qs=512, k=ADDR[1], ks=256, T=3, Hq=4, Hk=2, D=128, dt=0, wq=None, wk=None, eps=1e-6, pos=ADDR[2],
       f=ADDR[3], rot=128, il=0, qo=ADDR[4], ko=ADDR[5]):
    return L.attn_lib().nm_qk_norm_rope(q, qs, k, ks, T, Hq, Hk, D, dt, wq, wk, eps, pos, f, rot, il, qo, ko, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=2 ** 31), dict(Hq=-1), dict(Hk=65536), dict(D=0), dict(D=12), dict(D=520),
                                dict(rot=8), dict(rot=144), dict(rot=-16), dict(eps=-1e-6), dict(eps=math.inf),
                                dict(eps=math.nan), dict(qs=504), dict(qs=516), dict(ks=248), dict(ks=2 ** 31)])
def test_qk_bad_shape(kw):
    assert qk(**kw) == L.NM_ERR_BAD_SHAPE


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(pos=None), dict(f=None), dict(qo=None), dict(ko=None),
                                dict(q=ADDR[0] + 2), dict(k=ADDR[1] + 8), dict(qo=ADDR[4] + 4), dict(wq=ADDR[6] + 2),
                                dict(pos=ADDR[2] + 2), dict(qo=ADDR[0] + 16), dict(ko=ADDR[0]), dict(qo=ADDR[1]),
                                dict(ko=ADDR[4] + 1024), dict(wq=ADDR[4]), dict(qo=ADDR[2] - 16),
                                dict(qs=520, qo=ADDR[0]), dict(ko=ADDR[3] - 16)])
def test_qk_invalid_pointer(kw):
    assert qk(**kw) == L.NM_ERR_INVALID_ARG


def test_qk_dtype_and_empty():
    assert qk(dt=2) == L.NM_ERR_UNSUPPORTED
    assert qk(T=0) == L.NM_OK and qk(Hq=0, Hk=0) == L.NM_OK
    assert qk(T=0, q=None, k=None, pos=None, f=None, qo=None, ko=None) == L.NM_OK


def cache(**kw):
    d = dict(k=ADDR[8], v=ADDR[9], k_scale=ADDR[10], v_scale=ADDR[11], n_pages=4, page_size=16, heads=2, D=128, dtype=1,
             format=1)
    d.update(kw)
    return L.KvCacheStruct(**d)


def write(c, k=ADDR[0], ks=256, v=ADDR[1], vs=256, T=3, slots=ADDR[2]):
    return L.attn_lib().nm_kv_write(ctypes.byref(c) if c else None, k, ks, v, vs, T, slots, None)


def read(c, slots=ADDR[2], T=3, k=ADDR[0], v=ADDR[1]):
    return L.attn_lib().nm_kv_read(ctypes.byref(c) if c else None, slots, T, k, v, None)


def attn(c, q=ADDR[0], qs=512, B=3, Hq=4, pp=None, P=0, table=ADDR[1], stride=4, lens=ADDR[2], ml=64, scale=0.1, o=ADDR[3],
         lse=None, ws=ADDR[4], nb=1 << 24):
    return L.attn_lib().nm_attn_decode(q, qs, B, Hq, ctypes.byref(c) if c else None, pp, P, table, stride, lens, ml, scale,
                                       o, lse, ws, nb, None)


@pytest.mark.parametrize("call", (write, read, attn))
@pytest.mark.parametrize("kw,want", [(dict(dtype=2), 3), (dict(dtype=-1), 3), (dict(format=3), 3), (dict(format=-1), 3),
                                     (dict(n_pages=0), 2), (dict(page_size=24), 2), (dict(heads=0), 2), (dict(D=96), 2),
                                     (dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
                                     (dict(k=ADDR[8] + 8), 1), (dict(v_scale=ADDR[11] + 4), 1)])
def test_bad_caches(call, kw, want):
    assert call(cache(**kw)) == want
    assert call(None) == L.NM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,want", [(dict(T=-1), 2), (dict(T=2 ** 31), 2), (dict(ks=248), 2), (dict(vs=260), 2),
                                     (dict(k=None), 1), (dict(slots=None), 1), (dict(k=ADDR[0] + 2), 1),
                                     (dict(slots=ADDR[2] + 4), 1), (dict(k=ADDR[8]), 1), (dict(v=ADDR[8] + 256), 1),
                                     (dict(slots=ADDR[10] + 8), 1), (dict(T=0, k=None, v=None, slots=None), 0)])
def test_write_refusals(kw, want):
    assert write(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [(dict(T=-1), 2), (dict(k=None), 1), (dict(v=ADDR[1] + 8), 1), (dict(k=ADDR[1] + 16), 1),
                                     (dict(k=ADDR[9]), 1), (dict(v=ADDR[2] - 16), 1), (dict(v=ADDR[11]), 1),
                                     (dict(T=0, k=None, v=None, slots=None), 0)])
def test_read_refusals(kw, want):
    assert read(cache(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), 2), (dict(B=65536), 2), (dict(Hq=0), 2), (dict(Hq=5), 2), (dict(P=-1), 2), (dict(ml=-1), 2),
    (dict(P=2 ** 30 + 1), 2), (dict(ml=2 ** 30 + 1), 2), (dict(qs=504), 2), (dict(qs=516), 2), (dict(scale=math.nan), 2),
    (dict(scale=math.inf), 2), (dict(scale=-1.1e30), 2), (dict(stride=3), 2), (dict(B=65535, Hq=1026, qs=1026 * 128), 2),
    (dict(q=None), 1), (dict(o=None), 1), (dict(lens=None), 1), (dict(table=None), 1), (dict(P=5), 1), (dict(q=ADDR[0] + 2), 1),
    (dict(o=ADDR[3] + 8), 1), (dict(lens=ADDR[2] + 2), 1), (dict(ws=ADDR[4] + 16), 1), (dict(o=ADDR[0]), 1),
    (dict(lse=ADDR[3] + 64), 1), (dict(o=ADDR[8]), 1), (dict(ws=ADDR[10]), 1), (dict(lse=ADDR[2]), 1), (dict(nb=-1), 1),
    (dict(ws=ADDR[3]), 1), (dict(P=100000, pp=ADDR[5], ws=None), 1), (dict(P=100000, pp=ADDR[5], nb=1024), 1)])
def test_attention_refusals(kw, want):
    assert attn(cache(), **kw) == want


def test_attention_workspace_bytes():
    f = L.attn_lib().nm_attn_workspace_bytes
    assert f(1, 32, 8, 128, 0, 0, 40) == 0 and f(4, 8, 8, 64, 1, 0, 0) == 0
    assert f(32, 64, 8, 128, 2, 32768, 1024) > 0
    for bad in ((0, 8, 8, 64, 0, 0, 1), (1, 7, 2, 64, 0, 0, 1), (1, 8, 8, 80, 0, 0, 1), (1, 8, 8, 64, 0, -1, 1),
                (1, 8, 8, 64, 0, 0, 2 ** 31), (1, 8, 8, 64, 3, 0, 1), (1, 8, 8, 64, -1, 0, 1)):
        assert f(*bad) == -1


def test_python_refuses_host_tensors_and_formats():
    x = torch.zeros((1, 2, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        nm.qk_norm_rope(x, x, torch.zeros(1, dtype=torch.int32), torch.zeros(32))
    with pytest.raises(ValueError, match="format"):
        nm.KVCache(4, 16, 2, 64, torch.float16, "fp8", device="cpu")
    with pytest.raises(ValueError, match="no cache"):
        nm.KVCache(4, 15, 2, 64, torch.float16, device="cpu")
    with pytest.raises(TypeError, match="float16"):
        nm.KVCache(4, 16, 2, 64, torch.float32, device="cpu")
    with pytest.raises(TypeError, match="KVCache"):
        nm.kv_write(None, x, x, x)
    c = nm.KVCache(4, 16, 2, 64, torch.float16, device="cpu")      # a handle on host memory: no call takes it
    for f in (lambda: nm.kv_write(c, x, x, torch.zeros(1, dtype=torch.int64)), lambda: nm.kv_read(c, torch.zeros(1)),
              lambda: nm.attn_decode(x, c, None, torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(TypeError, match="CUDA"):
            f()


def test_python_refuses_sizes_that_ctypes_would_cut():
    for sizes in ((4, 2 ** 32 + 16, 2, 64), (2 ** 64 + 4, 16, 2, 64), (4, 16, 2 ** 32 + 2, 64), (4, 16, 2, 2 ** 32 + 64)):
        with pytest.raises(ValueError, match="no cache"):
            nm.KVCache(*sizes, torch.float16, device="cpu")
    c = nm.KVCache(4, 16, 2, 64, torch.float16, device="cpu")
    q, lens, pages = torch.zeros((1, 2, 64), dtype=torch.float16), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_len"):
        nm.attn_decode(q, c, pages.view(1, 1), lens, max_len=2000 - 2 ** 64)
    with pytest.raises(ValueError, match="prefix_len"):
        nm.attn_decode(q, c, None, lens, prefix_pages=pages, prefix_len=2000 - 2 ** 64)
