"""attn_tree on the GPU against the 64-bit formula: formats, types, widths, rows from one to several hundred, trees and
other masks, page sizes, ranges, unseen infinities and NaN; and all of a server's calls together."""
import math
import random

import numpy as np
import pytest
import torch

import attn_reference as ref
import serve_reference as sref
from sparse_matrix_vector_amd import inputs as I

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
FORMATS = ("16", "mx8", "mx4")


@pytest.fixture(scope="module")
def nm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_matrix_vector_amd as nm
    nm.lib()
    return nm


def rnd(shape, dtype, *tag, scale=1.0):
    g = torch.Generator().manual_seed(I.seed_of("tree", *tag) % (1 << 62))
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def tree(N, r):
    """Masks of a random tree of N drafts."""
    row = []
    for i in range(N):
        parent = r.randint(-1, i - 1)
        row.append((row[parent] if parent >= 0 else 0) | 1 << i)
    return row


def signed(masks):
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in masks], dtype=torch.int64, device="cuda")


class Case:
    """A cache that holds sequences of the given lengths (negative: padding) on shuffled pages, and their drafts."""

    def __init__(self, nm, fmt, dtype, D, heads, G, N, lens, page, masks=None, tag=0):
        self.nm, self.fmt, self.dtype, self.D, self.heads, self.G, self.N, self.lens = nm, fmt, dtype, D, heads, G, N, lens
        self.page, self.gone = page, {}
        r = random.Random(I.seed_of(fmt, D, N, tag, len(lens)))
        B, longest = len(lens), max(max(lens), 1)
        per = -(-longest // page)
        pages = [-(-max(n, 0) // page) for n in lens]
        order = list(range(sum(pages) + 3))
        r.shuffle(order)
        table, at = np.full((B, per), -1), 0
        for b, c in enumerate(pages):
            table[b, :c] = order[at:at + c]
            at += c
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda")
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.masks = masks or [tree(N, r) for _ in lens]
        self.visible = signed(self.masks)
        self.q = rnd((B, N, heads * G, D), dtype, "q", tag, scale=1.5)
        self.cache = nm.KVCache(len(order), page, heads, D, dtype, fmt)
        self.k, self.v, self.slots = [], [], []
        for b, n in enumerate(lens):
            n = max(n, 0)
            k, v = rnd((n, heads, D), dtype, "k", tag, b), rnd((n, heads, D), dtype, "v", tag, b)
            t = np.arange(n)
            self.slots.append(torch.tensor(table[b, t // page] * page + t % page, dtype=torch.int64, device="cuda"))
            nm.kv_write(self.cache, k, v, self.slots[-1])
            self.k.append(ref.quantised(ref.f64(k), fmt, dtype))
            self.v.append(ref.quantised(ref.f64(v), fmt, dtype))

    def widen(self, tokens=0):
        """A table wide enough (absent pages behind the lengths) that the plan takes the form that shares the cache."""
        rows = self.N * self.G
        tokens = max(tokens, (1 << 24) // (rows * len(self.lens) * self.heads) + 1)
        more = torch.full((len(self.lens), -(-tokens // self.page) - self.table.shape[1]), -1, dtype=torch.int32, device="cuda")
        self.table = torch.cat((self.table, more), 1)
        assert rows > 32 and self.table.shape[1] * self.page * len(self.lens) * self.heads * rows > 1 << 24
        return self

    def run(self, **kw):
        return self.nm.attn_tree(self.q, self.cache, self.table, self.lens_t, self.visible, **kw)

    def check(self, max_len=None, scale=None, rows=None, **kw):
        out, lse = torch.full_like(self.q, 7.0), torch.full(self.q.shape[:3], 7.0, device="cuda")
        self.run(max_len=max_len, scale=scale, out=out, lse=lse, **kw)
        q, got, got_l = ref.f64(self.q), ref.f64(out), ref.f64(lse)
        for b, n in enumerate(self.lens):
            if n < 0:
                assert (got[b] == 7).all() and (got_l[b] == 7).all()
                continue
            n = n if max_len is None else min(n, max_len)
            j = np.arange(n) - (n - self.N)
            for i in range(self.N) if rows is None else rows:
                bits = np.array([bool(self.masks[b][i] >> int(x) & 1) if x >= 0 else True for x in j], dtype=bool)
                bits[self.gone.get(b, [])] = False
                for h in range(self.heads):
                    at = slice(h * self.G, (h + 1) * self.G)
                    o, l, tol, ltol = sref.attend(q[b, i, at], self.k[b][:n, h], self.v[b][:n, h],
                                                  np.broadcast_to(bits, (self.G, n)),
                                                  self.D ** -0.5 if scale is None else scale, self.dtype, False)
                    sref.close(got[b, i, at], o, tol, ("o", b, i, h))
                    sref.close(got_l[b, i, at], l, ltol, ("lse", b, i, h))
        return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D,heads,G,N", [(64, 2, 1, 1), (64, 1, 4, 4), (128, 2, 4, 5), (128, 1, 4, 8), (128, 1, 3, 11),
                                         (64, 2, 2, 33), (128, 1, 8, 16), (64, 1, 8, 40), (256, 1, 4, 3), (256, 1, 2, 12),
                                         (256, 1, 4, 40)])
def test_shapes(nm, fmt, dtype, D, heads, G, N):
    """Every form of unit, lengths around the drafts, tiles and pages."""
    lens = [N, N + 1, 15 + N, 16 + N, 64, 100 + N, 130]
    Case(nm, fmt, dtype, D, heads, G, N, [max(n, N) for n in lens], 16, tag=D + N).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", (16, 32, 64, 128, 256))
def test_pages(nm, fmt, page):
    Case(nm, fmt, BF16, 64, 2, 2, 6, [200, 7, 63, 129, 257], page, tag=page).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D,G,N", [(64, 1, 3), (128, 4, 7), (128, 8, 9), (64, 8, 64), (256, 2, 20)])
def test_ranges(nm, fmt, D, G, N):
    """Long tokens cut into ranges that a second launch joins; drafts that lie across a border between ranges."""
    for n in (1024 + N // 2, 2500):
        Case(nm, fmt, F16, D, 1, G, N, [n, 300, 128 + N // 2, N], 64, tag=n).check(rows=sorted({0, N // 2, N - 1}))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D,heads,G,N", [(64, 2, 4, 9), (64, 1, 8, 64), (128, 1, 5, 7), (128, 2, 4, 16), (128, 1, 8, 9),
                                         (128, 1, 3, 43), (128, 1, 16, 16)])
def test_shared_form(nm, fmt, dtype, D, heads, G, N):
    """Row groups of every fullness in the form that shares the cache through LDS; short lengths, and several ranges."""
    lens = [N, N + 1, 15 + N, 16 + N, 64, 100 + N, 130, -1, 0]
    Case(nm, fmt, dtype, D, heads, G, N, [max(n, N) if n > 0 else n for n in lens], 16, tag=D + N).widen().check(
        rows=sorted({0, 1, N // 2, N - 1}))
    Case(nm, fmt, dtype, D, heads, G, N, [2500, 300, 1024 + N // 2, 5], 64, tag=N).widen().check(rows=sorted({0, N // 2, N - 1}))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,N", [(4, 16), (4, 27), (8, 40)])
def test_shared_form_in_one_range(nm, fmt, G, N):
    """So many sequences that none is cut: the units write the result."""
    r = random.Random(N)
    lens = [r.choice((-1, 0, N, N + r.randint(0, 90))) for _ in range(128)]
    Case(nm, fmt, BF16, 64, 4, G, N, lens, 16, tag=N).widen(1024).check(rows=(0, N - 1))


@pytest.mark.parametrize("dtype,D,G,N", [(BF16, 128, 4, 12), (F16, 64, 8, 20)])
@pytest.mark.parametrize("odd", (math.nan, math.inf))
def test_shared_form_unseen_infinities_and_nan(nm, dtype, D, G, N, odd):
    n = 150
    c = Case(nm, "16", dtype, D, 1, G, N, [n, n], 64, masks=[[1 << i for i in range(N)], tree(N, random.Random(3))]).widen()
    clean = c.run()
    bad = rnd((1, 1, D), dtype, "bad")
    bad[0, 0, 3] = odd
    for j in (0, N - 1):
        for b in (0, 1):
            at = c.slots[b][n - N + j:n - N + j + 1]
            k, v = nm.kv_read(c.cache, at)
            nm.kv_write(c.cache, k, bad, at)
            got = c.run()
            nm.kv_write(c.cache, torch.full_like(bad, odd), bad, at)    # keys, too
            got_k = c.run()
            nm.kv_write(c.cache, k, v, at)
            for i in range(N):
                if c.masks[b][i] >> j & 1:
                    assert not got[b, i, :, 3].isfinite().any()
                else:                                                   # another order of fp32 sums at most
                    for x in (got, got_k):
                        d = (x[b, i].double() - clean[b, i].double()).abs()
                        assert (d <= 2 * ref.UNIT[dtype] * (clean[b, i].double().abs() + 2.0 ** -10)).all()
            assert torch.equal(got[1 - b], clean[1 - b])
    assert torch.equal(c.run(), clean)


@pytest.mark.parametrize("fmt", FORMATS)
def test_shared_form_absent_pages(nm, fmt):
    c = Case(nm, fmt, F16, 64, 1, 4, 12, [300, 300, 90], 16).widen()
    c.table[0, 2], c.table[1, 18], c.table[1, 0], c.table[2, 0] = -5, 1 << 30, -1, 1 << 20
    c.gone = {0: np.r_[32:48], 1: np.r_[0:16, 288:300], 2: np.r_[0:16]}
    c.check()


def test_forms_agree_in_a_graph(nm):
    """One plan serves all lengths below max_len; lengths change between replays."""
    c = Case(nm, "mx4", F16, 128, 2, 4, 12, [1500, 700], 64).widen()
    ws, out = nm.attn_tree_workspace(2, 12, 8, c.cache, c.table.shape[1] * 64), torch.zeros_like(c.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, ws=ws)
    for n in (1500, 400, 33, 12):
        c.lens[0] = n
        c.lens_t[0] = n
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run())


def test_masks(nm):
    """Chains, stars, empty masks, all ones, bits behind the last draft."""
    N = 9
    chain = [(2 << i) - 1 for i in range(N)]
    star = [1 << i for i in range(N)]
    odd = [0, 2 ** 64 - 1, 1 << 63, 1 << 8, 0xAAAA, 0, 3, 1 << 9, 2 ** 63 - 1]
    for fmt in FORMATS:
        Case(nm, fmt, BF16, 64, 2, 2, N, [40, 9, 200], 16, masks=[chain, star, odd], tag=fmt).check()
    Case(nm, "16", F16, 128, 1, 2, 64, [64, 100, 512], 16, masks=[[(2 << i) - 1 for i in range(64)]] * 3).check()


def test_rows_that_see_nothing(nm):
    """No tokens before the drafts and an empty mask: zeros and -inf; also shorter than the drafts, and empty."""
    N = 5
    for D, G in ((64, 2), (128, 16)):
        c = Case(nm, "16", F16, D, 1, G, N, [5, 3, 0, 1, 20], 16, masks=[[0, 1, 0, 31, 16]] * 5)
        out = c.check()
        assert not out[2].any() and not out[0, 0].any()


def test_chain_is_decode(nm):
    """A chain's drafts are single tokens at increasing lengths."""
    N, n = 6, 333
    for fmt in FORMATS:
        c = Case(nm, fmt, BF16, 128, 2, 4, N, [n], 64, masks=[[(2 << i) - 1 for i in range(N)]], tag=fmt)
        got = c.run()
        lens = torch.arange(n - N + 1, n + 1, dtype=torch.int32, device="cuda")
        want = nm.attn_decode(c.q[0], c.cache, c.table.expand(N, -1).contiguous(), lens)
        assert ((got[0].double() - want.double()).abs() <= 2.0 ** -7 * (want.double().abs() + 2.0 ** -6)).all()


def test_padding_max_len_scale(nm):
    for D, G, N in ((64, 2, 5), (64, 8, 12), (256, 2, 20)):
        c = Case(nm, "mx8", BF16, D, 2, G, N, [70, -1, 300, -9, 40], 32, tag=D)
        c.check()
        c.check(max_len=100)
        c.check(max_len=0)
        for scale in (0.0, -0.2, 1.0):
            c.check(scale=scale, rows=(0, N - 1))


@pytest.mark.parametrize("dtype,D,G,N", [(F16, 64, 1, 6), (BF16, 128, 4, 6), (F16, 128, 8, 12), (BF16, 64, 8, 40),
                                         (F16, 256, 2, 6), (BF16, 256, 4, 12)])
@pytest.mark.parametrize("odd", (math.nan, math.inf))
def test_unseen_infinities_and_nan(nm, dtype, D, G, N, odd):
    """A draft that others do not see may hold anything; rows behind the last token too."""
    n, r = 150, random.Random(3)
    masks = [[1 << i for i in range(N)], tree(N, r)]
    c = Case(nm, "16", dtype, D, 1, G, N, [n, n], 64, masks=masks)
    clean = c.run()
    bad = rnd((1, 1, D), dtype, "bad")
    bad[0, 0, 3] = odd
    for j in (0, N // 2, N - 1):
        for b in (0, 1):
            at = c.slots[b][n - N + j:n - N + j + 1]
            k, v = nm.kv_read(c.cache, at)
            nm.kv_write(c.cache, k, bad, at)
            got = c.run()
            nm.kv_write(c.cache, k, v, at)
            for i in range(N):
                if masks[b][i] >> j & 1:
                    assert not got[b, i, :, 3].isfinite().any()
                    rest = [x for x in range(D) if x != 3]
                    assert got[b, i][:, rest].isfinite().all()
                else:                                                   # another order of fp32 sums at most
                    d = (got[b, i].double() - clean[b, i].double()).abs()
                    assert (d <= 2 * ref.UNIT[dtype] * (clean[b, i].double().abs() + 2.0 ** -10)).all()
            assert torch.equal(got[1 - b], clean[1 - b])
            nm.kv_write(c.cache, torch.full_like(bad, odd), bad, at)    # keys, too
            got = c.run()
            nm.kv_write(c.cache, k, v, at)
            for i in range(N):
                if not masks[b][i] >> j & 1:
                    assert got[b, i].isfinite().all()
    assert torch.equal(c.run(), clean)


def test_absent_pages(nm):
    """Page numbers outside the cache are not followed: their tokens count as absent."""
    c = Case(nm, "16", F16, 64, 1, 2, 4, [100, 100], 16)
    c.table[0, 2] = -5
    c.table[1, 6] = 1 << 30                                             # the drafts' page
    gone = np.r_[32:48]
    c.masks[1] = [0] * 4
    got = ref.f64(c.run())
    q = ref.f64(c.q)
    for i in range(4):
        seen = np.array([t < 96 or bool(c.masks[0][i] >> (t - 96) & 1) for t in range(100)])
        seen[gone] = False
        o, _, tol, _ = sref.attend(q[0, i], c.k[0][:, 0], c.v[0][:, 0], np.broadcast_to(seen, (2, 100)), 0.125, F16, False)
        sref.close(got[0, i], o, tol, i)
        o, _, tol, _ = sref.attend(q[1, i], c.k[1][:, 0], c.v[1][:, 0], np.broadcast_to(np.arange(100) < 96, (2, 100)), 0.125,
                                   F16, False)
        sref.close(got[1, i], o, tol, i)


def test_strided_and_empty(nm):
    c = Case(nm, "16", BF16, 64, 2, 2, 3, [50, 20], 16)
    want = c.run()
    wide = torch.zeros((2, 3, 4 * 64 + 40), dtype=BF16, device="cuda")
    q = wide[..., :256].unflatten(2, (4, 64))
    q.copy_(c.q)
    c.q = q
    assert torch.equal(c.run(), want)
    table = torch.zeros((2, 9), dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    c.table = table[:, :c.table.shape[1]]
    assert torch.equal(c.run(), want)
    none = nm.attn_tree(q[:0], c.cache, c.table[:0], c.lens_t[:0], c.visible[:0])
    assert none.shape == (0, 3, 4, 64)
    with pytest.raises(ValueError):
        nm.attn_tree(wide[..., :256].unflatten(2, (4, 64)).transpose(0, 1), c.cache, c.table.repeat(2, 1)[:3], c.lens_t,
                     c.visible)


def test_workspace_stream_and_graph(nm):
    c = Case(nm, "mx8", BF16, 128, 2, 4, 10, [1500, 700], 64)
    want = c.run()
    ws = nm.attn_tree_workspace(2, 10, 8, c.cache, c.table.shape[1] * 64)
    assert ws.numel() > 0
    ws.fill_(255)
    assert torch.equal(c.run(ws=ws), want)
    with pytest.raises(nm.NmError):
        c.run(ws=ws[:256])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out, ws=ws)
    for n in (1500, 400, 33):
        c.lens_t[0] = n
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.run())


def test_a_server_step(nm):
    """A prompt, a tree of drafts, their refusal and a token, with the book of pages: each call's numbers feed the next
    one, and what comes out is the formula's over the tokens that each sequence has."""
    B, hq, heads, D, page, dtype = 3, 4, 2, 64, 16, BF16
    cache, pages = nm.KVCache(40, page, heads, D, dtype), nm.KVPages(B, 12, 40, page)
    freq = torch.pow(10000.0, -torch.arange(32, device="cuda") / 32).float()
    K, V = [np.zeros((0, heads, D)) for _ in range(B)], [np.zeros((0, heads, D)) for _ in range(B)]

    def rows(n, tag):
        return [rnd((n, h, D), dtype, tag, i) for i, h in enumerate((hq, heads, heads))]

    def step(adds, n, tag):
        starts, slots, positions, granted = nm.kv_plan(pages, torch.tensor(adds, dtype=torch.int32, device="cuda"), n)
        q, k, v = rows(n, tag)
        q, k = nm.qk_norm_rope(q, k, positions, freq)
        nm.kv_write(cache, k, v, slots)
        s = starts.tolist()
        for b in range(B):
            K[b] = np.concatenate((K[b], ref.f64(k[s[b]:s[b + 1]])))
            V[b] = np.concatenate((V[b], ref.f64(v[s[b]:s[b + 1]])))
        return q, k, v, starts, granted

    q, k, v, starts, granted = step([50, 7, 0], 60, "prompt")            # three rows of padding
    assert granted.tolist() == [50, 7, 0]
    out = nm.attn_prompt(q, k, v, starts, out=torch.zeros_like(q))
    o, _, tol, _ = sref.prompt(ref.f64(q), ref.f64(k), ref.f64(v), starts.tolist(), starts.tolist(), D ** -0.5, dtype)
    sref.close(ref.f64(out[:57]), o[:57], tol[:57], "prompt")
    # a second piece of sequence 0 behind its first tokens, read back, beside a new prompt
    q, k, v, starts, granted = step([20, 0, 33], 53, "piece")
    held = torch.arange(70, device="cuda")
    slots0 = pages.table[0].long()[held // page] * page + held % page
    k0, v0 = nm.kv_read(cache, slots0)
    ks, vs = torch.cat((k0, k[20:])), torch.cat((v0, v[20:]))
    k_starts = torch.tensor([0, 70, 70, 103], dtype=torch.int32, device="cuda")
    out = nm.attn_prompt(q, ks, vs, starts, k_starts)
    o, _, tol, _ = sref.prompt(ref.f64(q), ref.f64(ks), ref.f64(vs), starts.tolist(), k_starts.tolist(), D ** -0.5, dtype)
    sref.close(ref.f64(out), o, tol, "piece")
    # a tree of four drafts each, of which the first chain of two is kept
    N, masks = 4, [1, 3, 5, 13]
    before = [len(x) for x in K]
    q, k, v, starts, granted = step([N] * B, N * B, "drafts")
    tq = q.view(B, N, hq, D)
    out = nm.attn_tree(tq, cache, pages.table, pages.lens, signed([masks] * B))
    for b in range(B):
        for i in range(N):
            seen = np.array([t < before[b] or bool(masks[i] >> (t - before[b]) & 1) for t in range(before[b] + N)])
            for h in range(heads):
                at = slice(2 * h, 2 * h + 2)
                o, _, tol, _ = sref.attend(ref.f64(tq[b, i, at]), K[b][:, h], V[b][:, h], np.broadcast_to(seen, (2, len(seen))),
                                           D ** -0.5, dtype, False)
                sref.close(ref.f64(out[b, i, at]), o, tol, ("draft", b, i, h))
    nm.kv_plan(pages, torch.full((B,), -2, dtype=torch.int32, device="cuda"), 0)
    K, V = [x[:-2] for x in K], [x[:-2] for x in V]
    # and a token each
    q, k, v, starts, granted = step([1] * B, B, "token")
    out = nm.attn_decode(q, cache, pages.table, pages.lens)
    assert pages.lens.tolist() == [len(x) for x in K]
    for b in range(B):
        o, _, tol, _ = ref.attend(ref.f64(q[b]), K[b], V[b], D ** -0.5, dtype)
        sref.close(ref.f64(out[b]), o, tol, ("token", b))
    # all end: every page is free again
    nm.kv_plan(pages, torch.full((B,), -1000, dtype=torch.int32, device="cuda"), 0)
    assert pages.n_free.item() == 40 and sorted(pages.free.tolist()) == list(range(40))
