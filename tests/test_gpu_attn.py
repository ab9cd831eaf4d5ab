"""The operators of include/nmattn.h on the GPU against 64-bit references:
per-head norm with rotation, the paged cache in its three formats, attention
with and without a shared prefix; then all of them together with the library's
products, as a decode layer uses them."""
import numpy as np
import pytest
import torch

import attn_reference as ref
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
    g = torch.Generator().manual_seed(I.seed_of("attn", *tag) % (1 << 62))
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def ints(n, lo, hi, *tag):
    g = torch.Generator().manual_seed(I.seed_of("ints", *tag) % (1 << 62))
    return torch.randint(lo, hi, (n,), generator=g)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def equal_values(got, want):
    """Exact values, NaN for NaN; a zero's sign is free."""
    return np.array_equal(ref.f64(got), want, equal_nan=True)


# ---- the cache ------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,D,heads,page,T", [(BF16, 128, 8, 64, 33), (F16, 64, 3, 16, 1), (F16, 256, 2, 32, 77),
                                                  (BF16, 64, 1, 128, 200), (F16, 128, 5, 256, 300),
                                                  (BF16, 256, 1, 16, 18)])
def test_cache_round_trip(nm, fmt, dtype, D, heads, page, T):
    pages = -(-T // page) + 3
    cache = nm.KVCache(pages, page, heads, D, dtype, fmt)
    k, v = (rnd((T, heads, D), dtype, n, D, T, scale=s) for n, s in (("k", 3.0), ("v", 0.02)))
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(5))[:T].cuda()
    nm.kv_write(cache, k, v, slots)
    gk, gv = nm.kv_read(cache, slots)
    assert equal_values(gk, ref.quantised(ref.f64(k), fmt, dtype, read=True))
    assert equal_values(gv, ref.quantised(ref.f64(v), fmt, dtype, read=True))
    # every other slot is as it was: zero
    rest = torch.tensor(sorted(set(range(pages * page)) - set(slots.tolist())), device="cuda")
    for t in nm.kv_read(cache, rest):
        assert not t.any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
def test_cache_every_word(nm, fmt, dtype):
    """All 65536 words, each in a block with words of nearby size (so that
    codes of every size occur) and again shuffled over all sizes."""
    words = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    order = torch.argsort(words.view(dtype).float().abs(), stable=True)
    for x in (words[order], words, words[torch.randperm(65536, generator=torch.Generator().manual_seed(3))]):
        rows = x.view(dtype).view(-1, 1, 128).cuda()
        T = rows.shape[0]
        cache = nm.KVCache(T // 64, 64, 1, 128, dtype, fmt)
        slots = torch.arange(T, device="cuda")
        nm.kv_write(cache, rows, rows.flip(0), slots)
        gk, gv = nm.kv_read(cache, slots)
        if fmt == "16":
            assert same(gk, rows) and same(gv, rows.flip(0))
        else:
            want = ref.quantised(ref.f64(rows), fmt, dtype, read=True)
            assert equal_values(gk, want)
            assert equal_values(gv, want[::-1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_cache_skips_and_keeps(nm, fmt):
    """Padding rows and slots behind the cache are skipped, everything else stays; reads outside give zeros."""
    cache = nm.KVCache(4, 16, 2, 64, BF16, fmt)
    k0, v0 = rnd((64, 2, 64), BF16, "k0"), rnd((64, 2, 64), BF16, "v0")
    nm.kv_write(cache, k0, v0, torch.arange(64, device="cuda"))
    k, v = rnd((6, 2, 64), BF16, "k1"), rnd((6, 2, 64), BF16, "v1")
    slots = torch.tensor([5, -1, 64, 63, -2 ** 40, 2 ** 40], device="cuda")
    nm.kv_write(cache, k, v, slots)
    k0[5], k0[63], v0[5], v0[63] = k[0], k[3], v[0], v[3]
    gk, gv = nm.kv_read(cache, torch.arange(64, device="cuda"))
    assert equal_values(gk, ref.quantised(ref.f64(k0), fmt, BF16))
    assert equal_values(gv, ref.quantised(ref.f64(v0), fmt, BF16))
    again = torch.tensor([5, 5, -1, 64, 2 ** 62], device="cuda")
    gk, gv = nm.kv_read(cache, again)
    assert same(gk[0], gk[1]) and gk[0].any() and not gk[2:].any() and not gv[2:].any()
    nm.kv_write(cache, k[:0], v[:0], slots[:0])
    assert nm.kv_read(cache, slots[:0])[0].shape == (0, 2, 64)


@pytest.mark.parametrize("fmt", FORMATS)
def test_cache_strided_rows(nm, fmt):
    T, heads, D = 21, 4, 128
    qkv = rnd((T, 10 * D + 8), F16, "fused")
    k, v = (qkv[:, a * D:(a + heads) * D].unflatten(1, (heads, D)) for a in (2, 6))
    a, b = (nm.KVCache(2, 16, heads, D, F16, fmt) for _ in range(2))
    slots = torch.arange(T, device="cuda")
    nm.kv_write(a, k, v, slots)
    nm.kv_write(b, k.contiguous(), v.contiguous(), slots)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    if fmt != "16":
        assert torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)


# ---- norm and rotation ------------------------------------------------------------

def frequencies(rot, base=10000.0):
    return torch.pow(base, -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1)).float().cuda()


@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("T,hq,hk,D,rot,norm,interleaved",
                         [(1, 32, 8, 128, 128, False, False), (1, 1, 1, 128, 128, True, True), (7, 40, 8, 128, 64, True, False),
                          (33, 5, 1, 64, 64, True, True), (3, 3, 2, 80, 32, True, False), (2, 9, 7, 96, 48, True, True),
                          (5, 2, 1, 256, 256, True, False), (4, 1, 1, 512, 512, True, False), (6, 3, 3, 8, 0, True, False),
                          (2, 7, 5, 16, 16, True, False), (3, 2, 2, 40, 32, False, True), (600, 3, 1, 128, 128, True, False),
                          (513, 2, 2, 64, 32, False, True)])
def test_qk(nm, dtype, T, hq, hk, D, rot, norm, interleaved):
    q, k = rnd((T, hq, D), dtype, "q", T, D, scale=3.0), rnd((T, hk, D), dtype, "k", T, D, scale=0.5)
    wq, wk = (rnd((D,), dtype, n, D) if norm else None for n in ("wq", "wk"))
    pos = ints(T, 0, 1 << 20, T, D).int().cuda()
    f = frequencies(rot)
    gq, gk = nm.qk_norm_rope(q, k, pos, f, wq, wk, eps=1e-5, interleaved=interleaved)
    ref.qk_close(gq, q, wq, np.float32(1e-5).astype(float), pos, f, interleaved)
    ref.qk_close(gk, k, wk, np.float32(1e-5).astype(float), pos, f, interleaved)


def test_qk_one_weight_far_and_negative_positions(nm):
    q, k = rnd((4, 2, 128), BF16, "q"), rnd((4, 2, 128), BF16, "k")
    w, f = rnd((128,), BF16, "w"), frequencies(128)
    pos = torch.tensor([0, -5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    gq, gk = nm.qk_norm_rope(q, k, pos, f, None, w)
    ref.qk_close(gq, q, None, 1e-6, pos, f, False)
    ref.qk_close(gk, k, w, float(np.float32(1e-6)), pos, f, False)
    # position 0 without a norm: the row itself
    assert same(gq[0], q[0])


def test_qk_strided_and_in_place(nm):
    T, hq, hk, D = 9, 6, 2, 128
    qkv = rnd((T, (hq + 2 * hk) * D), F16, "fused")
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    w, pos, f = rnd((D,), F16, "w"), torch.arange(T, device="cuda").int(), frequencies(D)
    gq, gk = nm.qk_norm_rope(q, k, pos, f, w, w)
    qc, kc = q.contiguous(), k.contiguous()
    assert nm.qk_norm_rope(qc, kc, pos, f, w, w, out=(qc, kc))[0] is qc
    assert same(gq, qc) and same(gk, kc)
    ref.qk_close(gq, q, w, float(np.float32(1e-6)), pos, f, False)


def test_qk_special_values(nm):
    """An infinity or NaN stays in its head (and, without a norm, in its pair); a zero head stays zero."""
    q = rnd((1, 4, 64), F16, "q")
    q[0, 0, 3], q[0, 1, 7], q[0, 2] = float("inf"), float("nan"), 0.0
    k, f = rnd((1, 1, 64), F16, "k"), frequencies(32)
    pos = torch.tensor([3], dtype=torch.int32, device="cuda")
    gq, gk = nm.qk_norm_rope(q, k, pos, f)
    bad = ~torch.isfinite(gq[0].cpu())
    assert set(bad[0].nonzero().flatten().tolist()) == {3, 19}
    assert set(bad[1].nonzero().flatten().tolist()) == {7, 23}
    assert not gq[0, 2].any() and not bad[2:].any()
    gq, gk = nm.qk_norm_rope(q, k, pos, f, torch.ones(64, dtype=F16, device="cuda"))
    assert not gq[0, 2].any() and torch.isfinite(gq[0, 2:]).all()


def test_qk_no_rows_no_heads(nm):
    f, pos = frequencies(64), torch.zeros(3, dtype=torch.int32, device="cuda")
    q, k = rnd((3, 2, 64), F16, "q"), rnd((3, 0, 64), F16, "k")
    gq, gk = nm.qk_norm_rope(q, k, pos, f)
    assert gk.shape == (3, 0, 64) and same(gq, q)
    gq, gk = nm.qk_norm_rope(q[:0], k[:0], pos[:0], f)
    assert gq.shape == (0, 2, 64)


def test_qk_more_rows_than_a_grid_dimension_holds(nm):
    """2^22 + 5 rows, a block each: the grid has a second row.  All rows alike but the first and the last ones."""
    T, D = (1 << 22) + 5, 16
    q = rnd((1, 1, D), F16, "many").expand(T, 1, D).contiguous()
    ends = torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, T - 1], device="cuda")
    q[ends] = rnd((5, 1, D), F16, "ends")
    pos, f, w = torch.full((T,), 7, dtype=torch.int32, device="cuda"), frequencies(16), rnd((D,), F16, "w")
    pos[ends] = torch.tensor([3, 4, 5, 6, 8], dtype=torch.int32, device="cuda")
    gq, _ = nm.qk_norm_rope(q, q[:, :0], pos, f, w)
    eps = float(np.float32(1e-6))
    ref.qk_close(gq[ends], q[ends], w, eps, pos[ends], f, False)
    ref.qk_close(gq[2:3], q[2:3], w, eps, pos[2:3], f, False)
    gq[ends] = gq[2].clone()
    assert (gq == gq[2]).all()


# ---- attention ------------------------------------------------------------------

class Batch:
    """A filled cache with its tables: a prefix of P tokens shared by all, lens[b] tokens of each sequence's own,
    pages in random order; keys and values as the cache holds them, on the host."""

    def __init__(self, nm, dtype, fmt, D, hq, heads, page, P, lens, tag=0, scale=1.0, spare=2, garbage=None):
        self.nm, self.dtype, self.fmt, self.P, self.lens, self.page = nm, dtype, fmt, P, lens, page
        counts = [-(-max(n, 0) // page) for n in lens]
        pp = -(-P // page)
        n_pages = pp + sum(counts) + spare
        order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(17 + tag))
        self.cache = nm.KVCache(n_pages, page, heads, D, dtype, fmt)
        if garbage is not None:
            every = torch.full((n_pages * page, heads, D), garbage, dtype=dtype, device="cuda")
            nm.kv_write(self.cache, every, every, torch.arange(n_pages * page, device="cuda"))
        self.prefix_pages = order[:pp].int().cuda()
        width = max(1, max(counts, default=1))
        table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)
        at, slots = pp, [order[torch.arange(P) // page] * page + torch.arange(P) % page]
        for b, c in enumerate(counts):
            table[b, :c] = order[at:at + c].int()
            i = torch.arange(max(lens[b], 0))
            slots.append(order[at + i // page] * page + i % page)
            at += c
        self.table, self.t_lens = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.slots = torch.cat(slots)
        n = self.slots.shape[0]
        self.k, self.v = rnd((n, heads, D), dtype, "ak", tag, D, scale=scale), rnd((n, heads, D), dtype, "av", tag, D)
        self.q = rnd((len(lens), hq, D), dtype, "aq", tag, D)
        nm.kv_write(self.cache, self.k, self.v, self.slots.cuda())
        self.qk, self.qv = (ref.quantised(ref.f64(t), fmt, dtype) for t in (self.k, self.v))

    def run(self, **kw):
        return self.nm.attn_decode(self.q, self.cache, self.table, self.t_lens, prefix_pages=self.prefix_pages,
                                   prefix_len=self.P, **kw)

    def tokens(self, b):
        at = self.P + sum(max(n, 0) for n in self.lens[:b])
        return list(range(self.P)) + list(range(at, at + max(self.lens[b], 0)))

    def check(self, o, lse=None, scale=None, drop=None):
        scale = 1.0 / np.sqrt(self.q.shape[-1]) if scale is None else scale
        for b, n in enumerate(self.lens):
            if n < 0:
                continue
            t = [i for i in self.tokens(b) if drop is None or i not in drop]
            want, wl, tol, ltol = ref.attend(ref.f64(self.q[b]), self.qk[t], self.qv[t], scale, self.dtype)
            err = np.abs(ref.f64(o[b]) - want)
            assert (err <= tol).all(), (b, n, float((err / tol).max()))
            if lse is not None:
                got = ref.f64(lse[b])
                assert np.array_equal(np.isinf(got), np.isinf(wl))
                fin = np.isfinite(wl)
                assert (np.abs(got[fin] - wl[fin]) <= ltol[fin]).all(), (b, got, wl)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D,hq,heads,page,P,lens", [
    (128, 4, 1, 16, 0, [1]), (128, 8, 8, 16, 0, [37]), (128, 32, 8, 64, 0, [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129]),
    (64, 10, 2, 32, 0, [300, 5]), (256, 6, 2, 16, 0, [100, 0, 64]), (128, 5, 1, 128, 0, [1000]),
    (64, 32, 1, 16, 0, [70, 3]), (128, 20, 1, 32, 0, [40, 257]),
    (128, 8, 2, 16, 40, [0, 3, 33]), (128, 8, 8, 64, 1, [0]), (64, 16, 2, 32, 161, [5] * 5), (128, 32, 8, 64, 300, [1, 0] * 6),
    (256, 8, 1, 16, 130, [7, 0, 50]), (128, 16, 2, 16, 515, [9] * 33), (64, 4, 4, 256, 257, [0, 0, -1, 2]),
    (256, 16, 2, 32, 100, [20] * 6)])
def test_attention(nm, dtype, fmt, D, hq, heads, page, P, lens):
    b = Batch(nm, dtype, fmt, D, hq, heads, page, P, lens)
    lse = torch.full((len(lens), hq), 7.0, device="cuda")
    o = torch.full((len(lens), hq, D), 3.0, dtype=dtype, device="cuda")
    assert b.run(out=o, lse=lse) is o
    b.check(o, lse)
    for i, n in enumerate(lens):                      # padding rows are left as they were
        if n < 0:
            assert (o[i] == 3.0).all() and (lse[i] == 7.0).all()
    assert same(o[[i for i, n in enumerate(lens) if n >= 0]], b.run()[[i for i, n in enumerate(lens) if n >= 0]])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("P,lens,hq", [(0, [5000], 8), (3000, [900, 20, 0], 8), (2049, [10] * 20, 16)])
def test_attention_long(nm, fmt, P, lens, hq):
    """Several ranges a row, joined by the second launch; peaked scores."""
    b = Batch(nm, BF16, fmt, 128, hq, 2, 64, P, lens, scale=4.0)
    lse = torch.empty((len(lens), hq), device="cuda")
    b.check(b.run(lse=lse), lse)


@pytest.mark.parametrize("scale", (0.0, -0.3, 2.5))
def test_attention_scale(nm, scale):
    b = Batch(nm, F16, "16", 64, 4, 2, 16, 20, [50, 3])
    b.check(b.run(scale=scale), scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("garbage", (float("nan"), float("inf"), -float("inf")))
def test_attention_unseen_tokens(nm, fmt, garbage):
    """NaN and infinities everywhere that no sequence looks: the rest of last pages, of the prefix's, other pages."""
    args = (nm, BF16, fmt, 128, 8, 2, 32, 45, [1, 0, 17, 40, 250])
    clean, dirty = Batch(*args), Batch(*args, garbage=garbage)
    o = dirty.run()
    dirty.check(o)
    assert same(o, clean.run())
    clean, dirty = Batch(*args[:7], 0, [3, 70]), Batch(*args[:7], 0, [3, 70], garbage=garbage)
    assert same(dirty.run(), clean.run())


# Rows of a key head that see the prefix: 48 and 160 of 128 columns, 48 of 256, 40 of 64.
SHARED = ((128, 4, 1, 12), (128, 10, 2, 32), (256, 8, 1, 6), (64, 20, 4, 8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D,hq,heads,B", SHARED)
def test_attention_shared_prefix(nm, dtype, fmt, D, hq, heads, B):
    """Prefixes of one token, around the 64 that are staged at a time, and of several ranges, own tokens beside them;
    with garbage wherever no sequence looks; a page of the prefix and one of a sequence outside the cache."""
    for i, P in enumerate((1, 63, 65, 200, 1500)):
        lens = [(7 * b + i) % 40 for b in range(B)]
        lens[1] = -1
        b = Batch(nm, dtype, fmt, D, hq, heads, 16, P, lens, tag=i)
        lse = torch.empty((B, hq), device="cuda")
        o = b.run(lse=lse)
        b.check(o, lse)
        dirty = Batch(nm, dtype, fmt, D, hq, heads, 16, P, lens, tag=i, garbage=(float("nan"), float("inf"))[i % 2])
        seen = [k for k, n in enumerate(lens) if n >= 0]
        assert same(dirty.run()[seen], o[seen])
    drop = set(range(32, 48)) | set(b.tokens(0)[1500:1516])
    dirty.prefix_pages[2] = -1
    dirty.table[0, 0] = dirty.cache.n_pages
    dirty.check(dirty.run(lse=lse), lse, drop=drop)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_shared_prefix_peaked(nm, fmt):
    """Scores of which few count, the largest ones late: the running maximum grows from step to step."""
    b = Batch(nm, BF16, fmt, 128, 16, 2, 32, 700, [50] * 20, scale=1.0)
    ramp = torch.linspace(0.2, 6, b.k.shape[0]).view(-1, 1, 1).cuda()
    b.k = (b.k.float() * ramp).to(BF16)
    nm.kv_write(b.cache, b.k, b.v, b.slots.cuda())
    b.qk = ref.quantised(ref.f64(b.k), fmt, BF16)
    lse = torch.empty((20, 16), device="cuda")
    b.check(b.run(lse=lse), lse)


@pytest.mark.parametrize("slope", (0.02, 0.1, 0.7, -0.1))
@pytest.mark.parametrize("dtype,fmt", ((F16, "16"), (BF16, "16"), (F16, "mx8"), (BF16, "mx4")))
@pytest.mark.parametrize("P,lens", ((0, [1000, 300, 40]), (900, [40, 90, 0] * 4)))
def test_attention_climbing_scores(nm, dtype, fmt, P, lens, slope):
    """Scores that rise (or fall) from token to token, less or more than e^5 a step of 32 or 64: references that lag
    behind the maximum, and weights above one."""
    b = Batch(nm, dtype, fmt, 128, 8, 2, 16, P, lens)
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = 1.0
    b.q[..., 1] = 0.125
    b.k[..., 0] = (slope * torch.arange(b.k.shape[0], device="cuda") % 200).view(-1, 1).to(dtype)
    nm.kv_write(b.cache, b.k, b.v, b.slots.cuda())
    b.qk = ref.quantised(ref.f64(b.k), fmt, dtype)
    lse = torch.empty((len(lens), 8), device="cuda")
    b.check(b.run(scale=1.0, lse=lse), lse, scale=1.0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
def test_attention_seen_nan_stays_in_its_rows(nm, dtype, fmt):
    b = Batch(nm, dtype, fmt, 128, 4, 2, 16, 0, [40, 40])
    k, v = b.k[3:4].clone(), b.v[3:4].clone()
    v[0, 1, 5] = float("nan")                         # token 3 of sequence 0, key head 1
    b.nm.kv_write(b.cache, k, v, b.slots[3:4].cuda())
    o = b.run()
    assert torch.isnan(o[0, 2:, 5]).all() and torch.isfinite(o[0, :2]).all() and torch.isfinite(o[1]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype,size", ((F16, 65504.0), (F16, 2.0 ** -13), (F16, 2.0 ** -20), (BF16, 2.0 ** 60),
                                        (BF16, 2.0 ** -60)))
@pytest.mark.parametrize("P,B", ((0, 2), (90, 12)))
def test_attention_large_and_small_values(nm, dtype, fmt, size, P, B):
    """Values at the ends of the type's range (fp16: up to its largest, whose codes stand for 65536), and keys as
    small; the operands of quantised caches hold all of them exactly."""
    b = Batch(nm, dtype, fmt, 128, 4, 1, 16, P, [20 + 3 * i for i in range(B)])
    b.v = (b.v.float().clamp(-1, 1) * size).to(dtype)
    if size < 1:
        b.k = (b.k.float() * size).to(dtype)
        b.q = (b.q.float() * (min(1 / size, 2.0 ** 12))).to(dtype)
    nm.kv_write(b.cache, b.k, b.v, b.slots.cuda())
    b.qk, b.qv = (ref.quantised(ref.f64(t), fmt, dtype) for t in (b.k, b.v))
    o = b.run()
    if size == 65504.0 and fmt != "16":                # a mean of 65536s is past fp16
        big = torch.isinf(o).cpu().numpy()
        o = o.clamp(-65504, 65504)
        assert big.mean() < 0.05
    b.check(o)


def test_attention_bad_pages(nm):
    """Page numbers outside the cache: their tokens are absent, for own pages and for the prefix's."""
    b = Batch(nm, F16, "mx8", 128, 8, 2, 16, 50, [40, 16, 33])
    drop = set()
    for row, col, bad in ((0, 1, -1), (1, 0, b.cache.n_pages), (2, 2, 2 ** 31 - 1)):
        b.table[row, col] = bad
        t = b.tokens(row)[b.P:]
        drop |= set(t[col * 16:(col + 1) * 16])
    b.prefix_pages[1] = -2 ** 31
    drop |= set(range(16, 32))
    lse = torch.empty((3, 8), device="cuda")
    b.check(b.run(lse=lse), lse, drop=drop)
    b.prefix_pages[:] = -1
    b.table[:] = b.cache.n_pages
    assert not b.run(lse=lse).any() and torch.isneginf(lse).all()


def test_attention_lens_beyond_max_len(nm):
    """A length above max_len counts as max_len."""
    b = Batch(nm, BF16, "16", 64, 4, 2, 16, 0, [48, 20])
    want = b.run()
    b.t_lens[0] = 2 ** 31 - 1
    assert same(b.run(), want)
    short = b.run(max_len=32)
    b.t_lens[0] = 32
    assert same(short, b.run())


def test_attention_strided_q_and_table(nm):
    b = Batch(nm, BF16, "mx4", 128, 8, 2, 16, 17, [40, 3, 100])
    want = b.run()
    wide = torch.zeros((3, 20 * 128), dtype=BF16, device="cuda")
    wide[:, 256:256 + 1024] = b.q.flatten(1)
    b.q = wide[:, 256:256 + 1024].unflatten(1, (8, 128))
    table = torch.full((3, b.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = b.table
    b.table = table[:, :b.table.shape[1]]
    assert same(b.run(), want)


def test_attention_prefix_alone(nm):
    """No table at all, and lens of zero: every sequence sees the prefix only."""
    b = Batch(nm, BF16, "mx8", 128, 8, 2, 16, 100, [0, 0])
    o = nm.attn_decode(b.q, b.cache, None, b.t_lens, prefix_pages=b.prefix_pages, prefix_len=100)
    b.check(o)
    assert not nm.attn_decode(b.q, b.cache, None, b.t_lens).any()


@pytest.mark.parametrize("fmt", ("16", "mx4"))
def test_attention_offsets_past_32_bits(nm, fmt):
    """A cache above 4 GiB a buffer (and, at 4 bits, above 2^32 elements), its last pages used."""
    heads, D, page = 16, 256, 256
    per = heads * page * D * (2 if fmt == "16" else 1) // (1 if fmt == "16" else 2)
    n_pages = (1 << 32) // per + 3 if fmt == "16" else (1 << 33) // (2 * per) + 3
    cache = nm.KVCache(n_pages, page, heads, D, BF16, fmt)
    n = 2 * page + 3
    pages = torch.tensor([n_pages - 1, 0, n_pages - 2], dtype=torch.int32)
    i = torch.arange(n)
    slots = (pages.long()[i // page] * page + i % page).cuda()
    k, v = rnd((n, heads, D), BF16, "bigk"), rnd((n, heads, D), BF16, "bigv")
    nm.kv_write(cache, k, v, slots)
    gk, gv = nm.kv_read(cache, slots)
    wk, wv = ref.quantised(ref.f64(k), fmt, BF16), ref.quantised(ref.f64(v), fmt, BF16)
    assert equal_values(gk, wk) and equal_values(gv, wv)
    q = rnd((1, heads, D), BF16, "bigq")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    o = nm.attn_decode(q, cache, pages[None].cuda(), lens)
    want, _, tol, _ = ref.attend(ref.f64(q[0]), wk, wv, 1 / 16, BF16)
    assert (np.abs(ref.f64(o[0]) - want) <= tol).all()


@pytest.mark.parametrize("P", (0, 17))
def test_attention_more_units_than_a_grid_dimension_holds(nm, P):
    """65535 sequences on 66 heads, 2^22 + 2^17 units, every sequence on the same page."""
    B, heads, D = 65535, 66, 64
    cache = nm.KVCache(4, 16, heads, D, F16, "mx8")
    k, v = rnd((40, heads, D), F16, "uk"), rnd((40, heads, D), F16, "uv")
    nm.kv_write(cache, k, v, torch.arange(40, device="cuda"))
    q = rnd((64, heads, D), F16, "uq")[torch.arange(B, device="cuda") % 64]
    lens = (torch.arange(B, device="cuda") % 5).int()
    table = torch.full((B, 1), 2, dtype=torch.int32, device="cuda")
    pages = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    o = nm.attn_decode(q, cache, table, lens, prefix_pages=pages, prefix_len=P)
    kk, vv = (ref.quantised(ref.f64(t), "mx8", F16) for t in (k, v))
    for b in (0, 1, 63549, 63550, 63551, 65534):          # around unit 2^22 and both ends
        t = list(range(P)) + list(range(32, 32 + int(lens[b])))
        want, _, tol, _ = ref.attend(ref.f64(q[b]), kk[t], vv[t], 0.125, F16)
        assert (np.abs(ref.f64(o[b]) - want) <= tol).all(), b
    assert same(o[:320], o[64960:65280])                  # the same queries and lengths come back every 320


# ---- streams, graphs, workspaces -----------------------------------------------------

def test_streams_at_once(nm):
    """The same calls on several streams at the same time, each with a workspace of its own or an allocated one."""
    batches = [Batch(nm, BF16, f, 128, 16, 2, 32, 300, [200, 5, 900], tag=i) for i, f in enumerate(FORMATS)]
    want = [b.run() for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = []
    for rep in range(3):
        for b, s in zip(batches, streams):
            ws = nm.attn_workspace(3, 16, b.cache, b.table.shape[1] * 32, 300) if rep else None
            got.append(b.run(stream=s, ws=ws))
            if ws is not None:
                ws.record_stream(s)
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert same(o, want[i % 3])


def test_graph_replays_with_new_inputs(nm):
    """A captured step (norm, write, attention): replayed with new rows, positions, slots and lengths, eager work
    and synchronisations between the replays; every replay equals the eager result."""
    dtype, heads, hq, D, page, B = BF16, 2, 8, 128, 16, 3
    a, e = (Batch(nm, dtype, "mx8", D, hq, heads, page, 40, [30, 47, 0], tag=1) for _ in range(2))
    w, f = rnd((D,), dtype, "w"), frequencies(D)
    q0, k0, v0 = (torch.zeros((B, n, D), dtype=dtype, device="cuda") for n in (hq, heads, heads))
    pos, slots = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), -1, device="cuda")
    tables = [torch.cat((x.table, torch.zeros((B, 1), dtype=torch.int32, device="cuda")), 1) for x in (a, e)]
    for x, t in zip((a, e), tables):
        t[:, 3] = torch.tensor([x.cache.n_pages - 1, 0, 1])
        x.table = t

    def step(x):
        q, k = nm.qk_norm_rope(q0, k0, pos, f, w, w)
        nm.kv_write(x.cache, k, v0, slots)
        return nm.attn_decode(q, x.cache, x.table, x.t_lens, max_len=64, prefix_pages=x.prefix_pages, prefix_len=40)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(a)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured = step(a)
    torch.cuda.synchronize()
    for rep in range(5):
        for t, n in ((q0, "q"), (k0, "k"), (v0, "v")):
            t.copy_(rnd(t.shape, dtype, n, rep))
        pos.copy_(torch.tensor([70 + rep, 87 + rep, -1]))
        own = torch.tensor([30 + rep, 47 + rep, 0])
        page_of = e.table[torch.arange(B), (own // page).cuda()].long().cpu()
        s = page_of * page + own % page
        s[2] = -1                                     # a padding row
        slots.copy_(s)
        for x in (a, e):
            x.t_lens.copy_(torch.tensor([31 + rep, 48 + rep, -1]))
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = step(e)
        assert same(captured[:2], eager[:2]), rep
        assert torch.equal(a.cache.k, e.cache.k) and torch.equal(a.cache.v, e.cache.v)
        del junk


def test_graph_of_a_shared_prefix(nm):
    """A captured call with staged prefix units, replayed with other queries and lengths."""
    b = Batch(nm, BF16, "mx8", 128, 16, 2, 32, 1000, [60] * 24, tag=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        b.run()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured = b.run()
    torch.cuda.synchronize()
    for rep in range(4):
        b.q.copy_(rnd(b.q.shape, BF16, "gq", rep))
        b.t_lens.copy_(ints(24, 0, 61, "gl", rep))
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(captured, b.run()), rep
        del junk


def test_two_graphs_share_a_workspace(nm):
    """Two captured calls with one workspace, replayed one after the other on one stream: no state is left in it."""
    a = Batch(nm, BF16, "16", 128, 8, 2, 64, 1500, [700, 3], tag=3)
    c = Batch(nm, F16, "mx4", 128, 8, 2, 32, 900, [2000], tag=4)
    need = [nm.attn_workspace(len(x.lens), 8, x.cache, x.table.shape[1] * x.page, x.P).numel() for x in (a, c)]
    assert min(need) > 0
    ws = torch.full((max(need),), 255, dtype=torch.uint8, device="cuda")      # any contents
    want = [a.run(), c.run()]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in (a, c):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(x.run(ws=ws))
            graphs.append(g)
        for rep in range(4):
            for i in (0, 1, 1, 0):
                outs[i].zero_()
                graphs[i].replay()
                torch.cuda.synchronize()
                assert same(outs[i], want[i]), (rep, i)


# ---- together -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype,fmt,norm", [(BF16, "mx8", True), (F16, "16", False), (BF16, "mx4", True)])
def test_decode_layer(nm, dtype, fmt, norm):
    """Several decode steps of a small layer's attention half, as a decoder runs it: q+k+v as one sparse product,
    norm and rotation, cache write, attention behind a shared prefix, the output projection; each operator checked
    on the inputs it had."""
    B, hidden, hq, heads, D, page, P = 3, 512, 8, 2, 128, 16, 37
    packs = [nm.pack(I.weight(n * D, hidden, dtype, I.seed_of("layer", i), sigma=0.1).cuda())
             for i, n in enumerate((hq, heads, heads))]
    o_pack = nm.pack(I.weight(hidden, hq * D, dtype, I.seed_of("layer", "o")).cuda())
    w = rnd((D,), dtype, "lw") if norm else None
    f = frequencies(D)
    cache = nm.KVCache(16, page, heads, D, dtype, fmt)
    order = torch.randperm(16, generator=torch.Generator().manual_seed(1))
    prefix_pages, table = order[:3].int().cuda(), order[3:9].view(3, 2).int().cuda()
    held = {}                                         # slot -> (k, v) as given to the cache

    def write(k, v, slots):
        nm.kv_write(cache, k, v, slots)
        for s, a, b in zip(slots.tolist(), ref.f64(k), ref.f64(v)):
            held[s] = (ref.quantised(a, fmt, dtype), ref.quantised(b, fmt, dtype))

    i = torch.arange(P)
    prefix_slots = (order[i // page] * page + i % page)
    x = rnd((P, hidden), dtype, "prompt")
    ks, vs = zip(*(nm.spmv_multi(packs[1:], x[a:a + 16]) for a in range(0, P, 16)))
    k, v = torch.cat(ks).view(P, heads, D), torch.cat(vs).view(P, heads, D)
    q_none = torch.empty((P, 0, D), dtype=dtype, device="cuda")
    _, k = nm.qk_norm_rope(q_none, k, i.int().cuda(), f, None, w)
    write(k, v, prefix_slots.cuda())
    for step in range(20):
        x = rnd((B, hidden), dtype, "x", step)
        q, k, v = (t.view(B, -1, D) for t in nm.spmv_multi(packs, x))
        pos = torch.full((B,), P + step, dtype=torch.int32, device="cuda")
        qr, kr = nm.qk_norm_rope(q, k, pos, f, w, w)
        eps = float(np.float32(1e-6))
        ref.qk_close(qr, q, w, eps, pos, f, False)
        ref.qk_close(kr, k, w, eps, pos, f, False)
        slots = table[:, step // page].long() * page + step % page
        write(kr, v, slots)
        lens = torch.full((B,), step + 1, dtype=torch.int32, device="cuda")
        o = nm.attn_decode(qr, cache, table, lens, prefix_pages=prefix_pages, prefix_len=P)
        if step in (0, 7, 19):
            for b in range(B):
                own = [int(table[b, t // page]) * page + t % page for t in range(step + 1)]
                seen = [held[s] for s in prefix_slots.tolist() + own]
                want, _, tol, _ = ref.attend(ref.f64(qr[b]), np.stack([s[0] for s in seen]),
                                             np.stack([s[1] for s in seen]), 1 / np.sqrt(D), dtype)
                assert (np.abs(ref.f64(o[b]) - want) <= tol).all(), (step, b)
        y = nm.spmv(*o_pack, o.view(B, hq * D))
        assert y.shape == (B, hidden) and torch.isfinite(y).all()
