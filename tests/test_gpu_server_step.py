"""A server's steps over the book of pages where some sequences get nothing (padding rows, rows of the table that are too
short, pages that run out): nm_kv_plan packs the new rows without gaps, the calls over a batch take sequence b's rows at
b N."""
import numpy as np
import pytest
import torch

import attn_reference as ref
import serve_reference as sref
from sparse_matrix_vector_amd import inputs as I

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
HQ, HEADS, D, PAGE = 4, 2, 64, 16
G = HQ // HEADS


@pytest.fixture(scope="module")
def nm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_matrix_vector_amd as nm
    nm.lib()
    return nm


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rnd(shape, dtype, *tag):
    g = torch.Generator().manual_seed(I.seed_of("server", *tag) % (1 << 62))
    return torch.randn(shape, generator=g).to(dtype).cuda()


def freq():
    return torch.pow(10000.0, -torch.arange(D // 2, device="cuda") / (D // 2)).float()


def in_batch(pages, starts, slots, granted, N):
    """What the calls over a batch take for N new tokens a sequence: slots [B][N] and lengths [B], -1 where a sequence got
    nothing."""
    rows = starts[:-1, None] + torch.arange(N, device="cuda")
    got = granted > 0
    return torch.where(got[:, None], slots[rows.clamp(max=len(slots) - 1)], -1), torch.where(got, pages.lens, -1)


class History:
    """What the cache holds of each sequence, in float64."""

    def __init__(self, B, fmt, dtype):
        self.fmt, self.dtype = fmt, dtype
        self.k = [np.zeros((0, HEADS, D)) for _ in range(B)]
        self.v = [np.zeros((0, HEADS, D)) for _ in range(B)]

    def add(self, b, k, v):
        self.k[b] = np.concatenate((self.k[b], ref.quantised(ref.f64(k), self.fmt, self.dtype)))
        self.v[b] = np.concatenate((self.v[b], ref.quantised(ref.f64(v), self.fmt, self.dtype)))

    def keep(self, b, which):
        self.k[b], self.v[b] = self.k[b][which], self.v[b][which]

    def check(self, b, q, out, seen, what, one_operand=False):
        """q and out [rows][HQ][D] of sequence b, seen [rows][tokens]."""
        for h in range(HEADS):
            at = slice(h * G, (h + 1) * G)
            for i in range(len(seen)):
                o, _, tol, _ = sref.attend(ref.f64(q[i, at]), self.k[b][:, h], self.v[b][:, h],
                                           np.broadcast_to(seen[i], (G, len(seen[i]))), D ** -0.5, self.dtype, one_operand)
                sref.close(ref.f64(out[i, at]), o, tol, (what, b, i, h))


@pytest.mark.parametrize("fmt,dtype", [("16", BF16), ("mx8", F16), ("mx4", BF16)])
def test_sequences_that_get_nothing(nm, fmt, dtype):
    """A tree step and a token step in which one sequence is a padding row, one's row of the table is too short and one
    finds no page left.  The others keep their own rows, and nothing is written for those."""
    B, N, masks, depth = 6, 4, [1, 3, 5, 13], [0, 1, 1, 2]
    held = [20, 0, 46, 7, 0, 15]
    pages, cache = nm.KVPages(B, 3, 8, PAGE), nm.KVCache(8, PAGE, HEADS, D, dtype, fmt)
    pages.lens[1] = -1
    past = History(B, fmt, dtype)

    # what they hold so far
    adds = list(held)
    adds[1] = 3                                                         # a padding row gets nothing
    starts, slots, positions, granted = nm.kv_plan(pages, i32(adds), 100)
    assert granted.tolist() == held
    k, v = (rnd((100, HEADS, D), dtype, n) for n in "kv")
    q, k = nm.qk_norm_rope(rnd((100, HQ, D), dtype, "q"), k, positions, freq())
    nm.kv_write(cache, k, v, slots)
    s = starts.tolist()
    for b in range(B):
        past.add(b, k[s[b]:s[b + 1]], v[s[b]:s[b + 1]])

    # a tree of four drafts each
    starts, slots, _, granted = nm.kv_plan(pages, i32([N] * B), B * N)
    assert granted.tolist() == [4, 0, 0, 4, 4, 0] and starts.tolist() == [0, 4, 4, 4, 8, 12, 12]
    slots, lens = in_batch(pages, starts, slots, granted, N)
    positions = (pages.lens[:, None] - N + i32(depth)).flatten()       # a draft's place in its text: its depth
    q, k, v = (rnd((B * N, h, D), dtype, n) for n, h in (("tq", HQ), ("tk", HEADS), ("tv", HEADS)))
    q, k = nm.qk_norm_rope(q, k, positions, freq())
    nm.kv_write(cache, k, v, slots.flatten())
    out = torch.full((B, N, HQ, D), 7.0, dtype=dtype, device="cuda")
    visible = torch.tensor([masks] * B, device="cuda")
    nm.attn_tree(q.view(B, N, HQ, D), cache, pages.table, lens, visible, out=out)
    for b, got in enumerate(granted.tolist()):
        if not got:
            assert (out[b] == 7).all()
            continue
        past.add(b, k[b * N:(b + 1) * N], v[b * N:(b + 1) * N])
        seen = np.array([[t < held[b] or bool(m >> (t - held[b]) & 1) for t in range(held[b] + N)] for m in masks])
        past.check(b, q.view(B, N, HQ, D)[b], out[b], seen, "draft")

    # drafts 0 and 2 are kept: the second kept one moves to its place, the rest go
    kept_k, kept_v = nm.kv_read(cache, slots[:, 2].contiguous())
    nm.kv_write(cache, kept_k, kept_v, slots[:, 1].contiguous())
    refused = torch.where(granted > 0, 2, 0).int()
    nm.kv_plan(pages, -refused, 0)
    for b, got in enumerate(granted.tolist()):
        if got:
            past.keep(b, list(range(held[b])) + [held[b], held[b] + 2])
    assert pages.lens.tolist() == [22, -1, 46, 9, 2, 15]

    # a token each; pages have come back in no case, so that the last one still has room on its page
    starts, slots, _, granted = nm.kv_plan(pages, i32([1] * B), B)
    assert granted.tolist() == [1, 0, 1, 1, 1, 1] and starts.tolist() == [0, 1, 1, 2, 3, 4, 5]
    slots, lens = in_batch(pages, starts, slots, granted, 1)
    q, k, v = (rnd((B, h, D), dtype, n) for n, h in (("dq", HQ), ("dk", HEADS), ("dv", HEADS)))
    q, k = nm.qk_norm_rope(q, k, pages.lens - 1, freq())
    nm.kv_write(cache, k, v, slots.flatten())
    out = torch.full((B, HQ, D), 7.0, dtype=dtype, device="cuda")
    nm.attn_decode(q, cache, pages.table, lens, out=out)
    for b, got in enumerate(granted.tolist()):
        if not got:
            assert (out[b] == 7).all()
            continue
        past.add(b, k[b:b + 1], v[b:b + 1])
        assert len(past.k[b]) == pages.lens[b].item()
        past.check(b, q[b:b + 1], out[b:b + 1], np.ones((1, len(past.k[b])), bool), "token")
