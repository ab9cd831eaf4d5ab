"""Prompts, whole ones and pieces behind earlier tokens, over the book of pages with the past read out of the cache: one
graph for any requests."""
import numpy as np
import pytest
import torch

import attn_reference as ref
from test_gpu_server_step import D, HEADS, HQ, PAGE, History, freq, i32, nm, rnd  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def prompt_step(nm, pages, cache, adds, q, k, v, room, out):  # noqa: F811
    """New rows of prompts, whole ones and pieces behind earlier tokens, up to `room` tokens of them and their past
    together: all on the device, with sizes that do not depend on the requests."""
    rows, B, width = q.shape[0], pages.sequences, pages.width
    starts, slots, positions, granted = nm.kv_plan(pages, adds, rows)
    q, k = nm.qk_norm_rope(q, k, positions, freq())
    nm.kv_write(cache, k, v, slots)
    # keys and values of every sequence with new rows, read out of the cache one after the other
    held = torch.where(granted > 0, pages.lens, 0)
    k_starts = torch.cat((held.new_zeros(1), held.cumsum(0, dtype=torch.int32)))
    t = torch.arange(room, dtype=torch.int32, device="cuda")
    b = torch.searchsorted(k_starts[1:], t, right=True).clamp(max=B - 1)
    place = t - k_starts[b]
    page = pages.table[b, (place // PAGE).clamp(max=width - 1)].long()
    old = torch.where(t < k_starts[-1], page * PAGE + place % PAGE, -1)
    k, v = nm.kv_read(cache, old)
    nm.attn_prompt(q, k, v, starts, k_starts, out=out)
    return q, k, v, starts, k_starts, granted


@pytest.mark.parametrize("fmt,dtype", [("16", F16), ("mx8", BF16)])
def test_pieces_in_one_graph(nm, fmt, dtype):  # noqa: F811
    """Replays with other requests equal the same calls made one by one, and the formula over what the cache holds."""
    B, width, rows, room = 4, 9, 120, 500
    books = [nm.KVPages(B, width, 30, PAGE) for _ in range(2)]
    caches = [nm.KVCache(30, PAGE, HEADS, D, dtype, fmt) for _ in range(2)]
    adds, x = i32([0] * B), [rnd((rows, h, D), dtype, "g", h, i) for i, h in enumerate((HQ, HEADS, HEADS))]
    outs = [torch.zeros((rows, HQ, D), dtype=dtype, device="cuda") for _ in range(2)]
    prompt_step(nm, books[0], caches[0], adds, *x, room, outs[0])       # what torch makes once; nobody asks for anything
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = prompt_step(nm, books[0], caches[0], adds, *x, room, outs[0])
    past = History(B, fmt, dtype)
    for i, request in enumerate(([50, 7, 0, 33], [20, 0, 60, 1], [-70, 64, 30, 0], [0, 0, 0, 0], [120, 0, 0, 0], [1, 1, -90, 1],
                                 [-1000, 50, 9, 2], [40, 16, 40, 16])):
        adds.copy_(i32(request))
        for j, (t, h) in enumerate(zip(x, (HQ, HEADS, HEADS))):
            t.copy_(rnd((rows, h, D), dtype, "again", i, j))
        for out in outs:
            out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want = prompt_step(nm, books[1], caches[1], adds, *x, room, outs[1])
        for a, b in zip((*got, outs[0], books[0].table, books[0].lens, books[0].free, books[0].n_free),
                        (*want, outs[1], books[1].table, books[1].lens, books[1].free, books[1].n_free)):
            assert torch.equal(a, b), request
        q, k, v, starts, k_starts, granted = got
        s, ks, granted = starts.tolist(), k_starts.tolist(), granted.tolist()
        assert ks[-1] <= room and sum(n > 0 for n in granted) == sum(n > 0 for n in request)
        for b in range(B):
            if granted[b] < 0:
                past.keep(b, slice(0, len(past.k[b]) + granted[b]))
            if granted[b] <= 0:
                assert ks[b] == ks[b + 1]
                continue
            # kv_read rounds to dtype what a quantised cache holds: exact for these values
            past.keep(b, slice(0, ks[b + 1] - ks[b] - granted[b]))
            new = slice(ks[b + 1] - granted[b], ks[b + 1])
            past.k[b], past.v[b] = (np.concatenate((old, ref.f64(t[new]))) for old, t in ((past.k[b], k), (past.v[b], v)))
            n = len(past.k[b])
            assert np.array_equal(past.k[b], ref.f64(k[ks[b]:ks[b + 1]])) and n == books[0].lens[b].item()
            seen = np.arange(n)[None, :] <= np.arange(granted[b])[:, None] + n - granted[b]
            at = slice(s[b], s[b + 1])
            past.check(b, q[at], outs[0][at], seen, "piece", True)
        assert (outs[0][s[-1]:] == 7).all()
