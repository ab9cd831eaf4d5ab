"""attn_prompt on the GPU against the 64-bit formula: lengths, head groups, widths, packed sequences and pieces of
prompts, strides, masked infinities and NaN, streams and graphs."""
import math

import numpy as np
import pytest
import torch

import attn_reference as ref
import serve_reference as sref
from sparse_matrix_vector_amd import inputs as I

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def nm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import sparse_matrix_vector_amd as nm
    nm.lib()
    return nm


def rnd(shape, dtype, *tag, scale=1.0):
    g = torch.Generator().manual_seed(I.seed_of("prompt", *tag) % (1 << 62))
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def starts_of(lengths, first=0):
    return torch.tensor(np.cumsum([first] + list(lengths)), dtype=torch.int32, device="cuda")


def check(nm, q, k, v, starts, k_starts=None, scale=None, **kw):
    dtype, D = q.dtype, q.shape[-1]
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    nm.attn_prompt(q, k, v, starts, k_starts, scale, out=out, lse=lse, **kw)
    s = starts.tolist()
    o, l, tol, ltol = sref.prompt(ref.f64(q), ref.f64(k), ref.f64(v), s, s if k_starts is None else k_starts.tolist(),
                                  D ** -0.5 if scale is None else scale, dtype)
    outside = np.isnan(o).all((1, 2))
    got, got_l = ref.f64(out), ref.f64(lse)
    assert (got[outside] == 7).all() and (got_l[outside] == 7).all()          # rows of no sequence stay
    sref.close(got[~outside], o[~outside], tol[~outside], "o")
    sref.close(got_l[~outside], l[~outside], ltol[~outside], "lse")
    # without lse the same rows, bit for bit
    again = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    nm.attn_prompt(q, k, v, starts, k_starts, scale, out=again, **kw)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))
    return out


@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D", (64, 128, 256))
@pytest.mark.parametrize("n", (1, 2, 31, 32, 33, 63, 64, 65, 100, 129, 257))
def test_one_prompt(nm, dtype, D, n):
    q, k, v = rnd((n, 4, D), dtype, "q", n, D, scale=1.5), rnd((n, 2, D), dtype, "k", n, D), rnd((n, 2, D), dtype, "v", n, D)
    check(nm, q, k, v, starts_of([n]))


@pytest.mark.parametrize("hq,heads", [(1, 1), (3, 1), (5, 5), (6, 2), (40, 8), (20, 4), (33, 1), (300, 1)])
def test_head_groups(nm, hq, heads):
    n = 37 if hq < 100 else 5
    q, k, v = (rnd((n, h, 64), BF16, "g", hq, h, i) for i, h in enumerate((hq, heads, heads)))
    check(nm, q, k, v, starts_of([n]))


@pytest.mark.parametrize("dtype,D,hq,heads", [(BF16, 128, 8, 2), (F16, 64, 6, 2), (F16, 256, 3, 1), (BF16, 256, 4, 2)])
@pytest.mark.parametrize("lengths", [(1, 1, 1), (5, 0, 70, 33, 0, 1), (0, 0, 3), (130, 257, 64, 1, 63)])
def test_packed(nm, dtype, D, hq, heads, lengths):
    T = sum(lengths)
    q, k, v = (rnd((T, h, D), dtype, "p", T, i) for i, h in enumerate((hq, heads, heads)))
    check(nm, q, k, v, starts_of(lengths))


def test_many_sequences(nm):
    """More sequences than a wave looks at in one and in two turns."""
    for B in (64, 65, 200, 4200):
        g = np.random.default_rng(B)
        lengths = g.integers(0, 3, B)
        T = int(lengths.sum())
        q, k, v = (rnd((T, h, 64), F16, "m", B, i) for i, h in enumerate((2, 1, 1)))
        check(nm, q, k, v, starts_of(lengths))


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (F16, 256)])
@pytest.mark.parametrize("pieces", [[(1, 200)], [(33, 97)], [(7, 7), (1, 1), (20, 300), (64, 128)], [(5, 3), (0, 4), (40, 1)],
                                    [(3, 0), (2, 2)], [(100, 37)], [(1, 700), (130, 650)]])
def test_pieces(nm, dtype, D, pieces):
    """Keys before the queries; fewer keys than queries, so that the first rows see nothing."""
    nq, nk = zip(*pieces)
    q, k, v = (rnd((n, h, D), dtype, "c", n, i) for i, (n, h) in enumerate(((sum(nq), 4), (sum(nk), 2), (sum(nk), 2))))
    check(nm, q, k, v, starts_of(nq), starts_of(nk))


def test_gaps_and_bad_bounds(nm):
    """Rows before the first and behind the last sequence stay; bounds outside count as the nearest, a sequence that
    ends before it starts as empty."""
    q, k, v = rnd((50, 2, 64), BF16, 1), rnd((60, 1, 64), BF16, 2), rnd((60, 1, 64), BF16, 3)
    check(nm, q, k, v, starts_of([10, 20], first=3), starts_of([15, 20], first=10))
    a = nm.attn_prompt(q, k, v, starts_of([47], first=3), starts_of([50], first=10))
    b = nm.attn_prompt(q, k, v, starts_of([900], first=3), starts_of([9000], first=10))
    assert torch.equal(a[3:], b[3:])
    out = torch.full_like(q, 7.0)
    nm.attn_prompt(q, k, v, torch.tensor([20, 10], dtype=torch.int32, device="cuda"), starts_of([60]), out=out)
    assert (out == 7).all()
    nm.attn_prompt(q, k, v, starts_of([0, 0, 0]), starts_of([60, 0, 0]), out=out)
    assert (out == 7).all()
    nm.attn_prompt(q, k, v, starts_of([50]), torch.tensor([40, 20], dtype=torch.int32, device="cuda"), out=out)
    assert (out == 0).all()                                             # no keys


@pytest.mark.parametrize("tk", (200, 9000))
def test_starts_that_decrease(nm, tk):
    """No rows are written but those of o and lse, with and without ranges of keys."""
    q = torch.cat([rnd((200, 8, 64), BF16, i) for i in range(3)])[200:400]
    k, v = rnd((tk, 1, 64), BF16, 2), rnd((tk, 1, 64), BF16, 3)
    for starts in ([0, 100, 120, 10, 200], [5, 200, 0, 200, 0], [200, 190, 180, 5, 6, 7], [0, 180, 20, 30, 40, 0, 200, 1]):
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        out, lse = torch.full((600, 8, 64), 7.0, dtype=BF16, device="cuda"), torch.full((600, 8), 7.0, device="cuda")
        nm.attn_prompt(q, k, v, st, starts_of([tk] + [0] * (len(starts) - 2)), out=out[200:400], lse=lse[200:400])
        for t in (out, lse):
            assert (t[:200] == 7).all() and (t[400:] == 7).all()


def test_no_rows(nm):
    q, k = torch.empty((0, 4, 64), dtype=F16, device="cuda"), torch.empty((0, 2, 64), dtype=F16, device="cuda")
    assert nm.attn_prompt(q, k, k, starts_of([0])).shape == (0, 4, 64)
    assert nm.attn_prompt(q, k, k, starts_of([])).shape == (0, 4, 64)
    q = rnd((3, 4, 64), F16, 0)
    assert (nm.attn_prompt(q, k, k, starts_of([3]), starts_of([0])) == 0).all()


@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 64)])
def test_strided_rows(nm, dtype, D):
    T, hq, heads = 71, 6, 2
    qkv = rnd((T, (hq + 2 * heads) * D + 24), dtype, "fused")
    cut = [qkv[:, a * D:(a + n) * D].unflatten(1, (n, D)) for a, n in ((0, hq), (hq, heads), (hq + heads, heads))]
    whole = check(nm, *cut, starts_of([30, 41]))
    assert torch.equal(whole, nm.attn_prompt(*(t.contiguous() for t in cut), starts_of([30, 41])))
    one = [t[:1] for t in cut]                                          # a single row's stride is not looked at
    check(nm, *one, starts_of([1]))


@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("scale", (0.0, -0.3, 1e-3, 3.0))
def test_scales(nm, dtype, scale):
    q, k, v = (rnd((90, h, 64), dtype, "s", i) for i, h in enumerate((2, 1, 1)))
    check(nm, q, k, v, starts_of([90]), scale=scale)


@pytest.mark.parametrize("dtype", (F16, BF16))
def test_rising_and_falling_scores(nm, dtype):
    """Maxima that grow along the keys (the reference is raised again and again) and ones that fall."""
    n, D = 300, 64
    q = torch.full((n, 1, D), 1.0, dtype=dtype, device="cuda")
    v = rnd((n, 1, D), dtype, "v")
    for sign in (1, -1):
        ramp = (sign * torch.arange(n, device="cuda") * 0.25).to(dtype)
        k = (rnd((n, 1, D), dtype, "k", scale=0.05).float() + ramp[:, None, None].float() / D).to(dtype)
        check(nm, q, k, v, starts_of([n]), scale=1.0)


@pytest.mark.parametrize("dtype", (F16, BF16))
def test_large_values(nm, dtype):
    """Values at the end of the type's range come out as they are where all are alike."""
    n, D = 130, 64
    top = torch.finfo(dtype).max
    q, k = rnd((n, 2, D), dtype, 1), rnd((n, 1, D), dtype, 2)
    v = torch.full((n, 1, D), top, dtype=dtype, device="cuda")
    out = nm.attn_prompt(q, k, v, starts_of([n]), scale=1e-3).double()          # no sum of weights above 1
    assert ((out - top).abs() <= top * 2 * ref.UNIT[dtype]).all()


def reordered(got, want, v):
    """Equal but for the order of the fp32 sums.  A step with infinities or NaN among its values adds them up key by
    key: the terms w v are the same, two orders of n of them differ by at most 2 n 2^-24 of the sum of |w v| over the sum
    of w, which is at most max |v|; then both are rounded, half a step each."""
    got, want = got.double(), want.double()
    near = 2 * max(150, v.shape[0]) * 2.0 ** -24 * v[v.isfinite()].double().abs().max()
    unit = ref.UNIT[v.dtype]
    return bool(((got - want).abs() <= near + unit * (2 * want.abs() + near) + 2 * ref.TINY[v.dtype]).all())


@pytest.mark.parametrize("dtype,D", [(F16, 128), (BF16, 64), (BF16, 256)])
@pytest.mark.parametrize("odd", (math.nan, math.inf, -math.inf))
def test_unseen_infinities_and_nan(nm, dtype, D, odd):
    """What stands in a key or value does not reach the queries before it, nor another sequence."""
    n, at = 150, (0, 1, 37, 63, 64, 100, 149)
    q, k, v = (rnd((2 * n, h, D), dtype, "n", i, D) for i, h in enumerate((4, 2, 2)))
    st = starts_of([n, n])
    clean = nm.attn_prompt(q, k, v, st)
    for j in at:
        for t in (k, v):
            old = t[j].clone()
            t[j, 1, 5] = odd
            got = nm.attn_prompt(q, k, v, st)
            t[j] = old
            assert reordered(got[:j], clean[:j], v) and torch.equal(got[n:], clean[n:])
            assert torch.equal(got[:, :2], clean[:, :2])                # the other key head
            if t is v:                                                  # its column alone, of every later row
                assert not got[j:n, 2:, 5].isfinite().any()
                rest = [c for c in range(D) if c != 5]
                assert reordered(got[:n, 2:, rest], clean[:n, 2:, rest], v)
            elif math.isnan(odd):
                assert got[j:n, 2:].isnan().all()
    # in keys and values at once, as an unwritten row may hold anything
    k[100:n] = odd
    v[100:n] = odd
    got = nm.attn_prompt(q, k, v, st)
    assert reordered(got[:100], clean[:100], v) and torch.equal(got[n:], clean[n:])


def test_scores_of_minus_infinity(nm):
    """A key whose score is -inf weighs nothing; a row with no other keys gets zeros."""
    q = torch.ones((3, 1, 64), dtype=F16, device="cuda")
    k = torch.zeros((3, 1, 64), dtype=F16, device="cuda")
    k[0, 0, 0] = -math.inf
    v = rnd((3, 1, 64), F16, 1)
    lse = torch.empty((3, 1), device="cuda")
    out = nm.attn_prompt(q, k, v, starts_of([3]), lse=lse)
    assert (out[0] == 0).all() and lse[0, 0] == -math.inf
    assert torch.equal(out[1], v[1])


def test_far_rows(nm):
    """Rows more than 2^32 bytes into the buffers."""
    D, rows = 128, (1 << 24) + 300
    k, v = (torch.empty((rows, 1, D), dtype=F16, device="cuda") for _ in range(2))
    q = rnd((200, 2, D), F16, 1)
    k[-200:], v[-200:] = rnd((200, 1, D), F16, 2), rnd((200, 1, D), F16, 3)
    st = torch.tensor([rows - 200, rows], dtype=torch.int32, device="cuda")

    def same(out, qq, kk, vv):
        n = qq.shape[0]
        o, _, tol, _ = sref.prompt(ref.f64(qq), ref.f64(kk), ref.f64(vv), [0, n], [0, n], D ** -0.5, F16)
        sref.close(ref.f64(out), o, tol, "far")

    same(nm.attn_prompt(q, k, v, starts_of([200]), st), q, k[-200:], v[-200:])
    # and of widely strided rows
    big = torch.empty((40, 1 << 27), dtype=F16, device="cuda")
    kk = big[:, 64:64 + D].unflatten(1, (1, D))
    kk.copy_(k[-40:])
    vv = big[:, 1024:1024 + D].unflatten(1, (1, D))
    vv.copy_(v[-40:])
    same(nm.attn_prompt(q[-40:], kk, vv, starts_of([40])), q[-40:], k[-40:], v[-40:])


@pytest.mark.parametrize("dtype,D,hq,heads", [(BF16, 128, 4, 1), (F16, 64, 3, 3), (F16, 256, 2, 1)])
@pytest.mark.parametrize("pieces", [[(1, 5000)], [(40, 3001), (7, 20), (0, 900), (3, 2)], [(130, 4097)]])
def test_few_rows_behind_many_keys(nm, dtype, D, hq, heads, pieces):
    """Keys cut into ranges that a second launch joins; some sequences shorter than the ranges are many."""
    nq, nk = zip(*pieces)
    q, k, v = (rnd((n, h, D), dtype, "few", n, i) for i, (n, h) in enumerate(((sum(nq), hq), (sum(nk), heads), (sum(nk), heads))))
    ws = nm.attn_prompt_workspace(sum(nq), sum(nk), len(nq), hq, heads, D)
    assert ws.numel() > 0
    ws.fill_(255)
    out = check(nm, q, k, v, starts_of(nq), starts_of(nk), ws=ws)
    assert torch.equal(out, nm.attn_prompt(q, k, v, starts_of(nq), starts_of(nk)))
    with pytest.raises(nm.NmError):
        nm.attn_prompt(q, k, v, starts_of(nq), starts_of(nk), ws=ws[:256])


def test_masked_in_ranges(nm):
    """NaN and infinities behind the rows' last keys, in the last of many ranges; zeros where no range has a key."""
    q, k, v = rnd((20, 2, 64), BF16, "r"), rnd((4000, 1, 64), BF16, "k"), rnd((4000, 1, 64), BF16, "v")
    clean = nm.attn_prompt(q, k, v, starts_of([20]), starts_of([4000]))
    k[3990:] = math.nan
    v[3990:] = math.inf
    got = nm.attn_prompt(q, k, v, starts_of([20]), starts_of([4000]))
    assert got[:10].isfinite().all() and reordered(got[:10], clean[:10], v[:3990])
    assert not got[10:].isfinite().any()
    out = torch.full_like(q, 7.0)
    nm.attn_prompt(q, k[:3000], v[:3000], starts_of([20]), starts_of([0]), out=out)
    assert not out.any()


def test_long_prompt_rows(nm):
    """Rows of a long prompt against the formula, and against the same rows as a piece."""
    n, hq, heads, D = 4100, 4, 1, 128
    q, k, v = (rnd((n, h, D), BF16, "long", i) for i, h in enumerate((hq, heads, heads)))
    out = nm.attn_prompt(q, k, v, starts_of([n]))
    for i in (0, 63, 64, 1000, 2047, 4098, 4099):
        o, _, tol, _ = sref.prompt(ref.f64(q[i:i + 1]), ref.f64(k[:i + 1]), ref.f64(v[:i + 1]), [0, 1], [0, i + 1],
                                   D ** -0.5, BF16)
        sref.close(ref.f64(out[i:i + 1]), o, tol, i)


def test_stream_and_graph(nm):
    q, k, v = (rnd((200, h, 64), F16, "st", i) for i, h in enumerate((4, 2, 2)))
    st = starts_of([120, 80])
    want = nm.attn_prompt(q, k, v, st)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = nm.attn_prompt(q, k, v, st, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nm.attn_prompt(q, k, v, st, out=out)
    for i in range(3):
        q.copy_(rnd((200, 4, 64), F16, "st again", i))
        st.copy_(starts_of([10 + 50 * i, 190 - 50 * i]))                 # lengths may change between replays
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nm.attn_prompt(q, k, v, st))


def test_ranges_in_a_graph_and_on_two_streams(nm):
    """The second launch reads what this call's first wrote: replays with other lengths, and two calls at once."""
    q, k, v = rnd((24, 4, 128), BF16, "rg", 0), rnd((6000, 1, 128), BF16, "rg", 1), rnd((6000, 1, 128), BF16, "rg", 2)
    st, kst = starts_of([8, 16]), starts_of([5000, 1000])
    ws, out = [nm.attn_prompt_workspace(24, 6000, 2, 4, 1, 128) for _ in range(2)], torch.zeros_like(q)
    assert ws[0].numel() > 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nm.attn_prompt(q, k, v, st, kst, out=out, ws=ws[0])
    for n, nk in ((8, 5000), (1, 64), (24, 6000), (0, 0)):
        st.copy_(starts_of([n, 24 - n]))
        kst.copy_(starts_of([nk, 6000 - nk]))
        ws[0].fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, nm.attn_prompt(q, k, v, st, kst))
    q2, out2 = rnd((24, 4, 128), BF16, "rg", 3), torch.zeros_like(q)
    want = nm.attn_prompt(q, k, v, st, kst), nm.attn_prompt(q2, k, v, st, kst)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        nm.attn_prompt(q, k, v, st, kst, out=out, ws=ws[0], stream=streams[0])
        nm.attn_prompt(q2, k, v, st, kst, out=out2, ws=ws[1], stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(out2, want[1])
