"""Calls of nm_attn_decode that take other ways through its launch plan than the shapes of test_gpu_attn.py."""
import pytest
import torch

import attn_reference as ref
from test_gpu_attn import BF16, F16, FORMATS, Batch, nm, same  # noqa: F401  (nm: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_workspace_for_every_smaller_call(nm, fmt):  # noqa: F811
    """A workspace for the longest call, filled with ones, serves shorter and smaller ones; same results as without."""
    b = Batch(nm, BF16, fmt, 128, 8, 2, 64, 2000, [8100, 30, 0, 700])
    ws = nm.attn_workspace(4, 8, b.cache, 8193, 2000)
    every = b.t_lens.clone()
    for n, max_len, P in ((4, 8128, 2000), (1, 8128, 2000), (1, 8064, 0), (3, 513, 0), (2, 600, 1), (4, 0, 1999), (4, 128, 130)):
        ws.fill_(255)
        kw = dict(max_len=max_len, prefix_pages=b.prefix_pages, prefix_len=P)
        o = nm.attn_decode(b.q[:n], b.cache, b.table[:n], every[:n], ws=ws, **kw)
        assert same(o, nm.attn_decode(b.q[:n], b.cache, b.table[:n], every[:n], **kw)), (n, max_len, P)


def ask(b):
    lse = torch.full(b.q.shape[:2], 7.0, device="cuda")
    o = torch.full_like(b.q, 3.0)
    b.run(out=o, lse=lse)
    b.check(o, lse)
    assert same(o, b.run(out=torch.full_like(b.q, 3.0)))
    for i, n in enumerate(b.lens):
        if n < 0:
            assert (o[i] == 3.0).all() and (lse[i] == 7.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D,G,heads,P,lens", ((128, 17, 1, 300, [1500, 40]), (128, 20, 2, 0, [1500, 40]), (64, 33, 1, 300, [1500, 0, 40]),
                                              (64, 20, 1, 0, [700, -1, 1500]), (256, 17, 2, 130, [600, 40]), (256, 40, 1, 0, [40, 900])))
def test_many_query_heads_in_several_ranges(nm, dtype, fmt, D, G, heads, P, lens):  # noqa: F811
    """More than 16 query heads a key head, whose rows lie in row groups of 16 that tiles of the joining launch cross,
    with own tokens in several ranges."""
    ask(Batch(nm, dtype, fmt, D, G * heads, heads, 16, P, lens))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("B,G", ((5, 4), (8, 4), (1, 20), (1, 32), (17, 1)))
@pytest.mark.parametrize("P", (1, 1500))
def test_two_row_tiles_behind_a_prefix(nm, dtype, fmt, D, B, G, P):  # noqa: F811
    """17 to 32 rows of a key head: prefix units of two row tiles a wave that read the cache themselves, the second
    tile whole or in part; one range and several; own tokens beside them, a padding row."""
    lens = [(11 * b + P) % 45 for b in range(B)]
    if B > 1:
        lens[1] = -1
    ask(Batch(nm, dtype, fmt, D, 2 * G, 2, 32, P, lens))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D,B,G,heads", ((128, 12, 4, 1), (64, 12, 4, 1), (128, 10, 16, 1), (64, 20, 8, 2), (256, 12, 4, 1)))
def test_staged_prefix_beside_long_own_tokens(nm, dtype, fmt, D, B, G, heads):  # noqa: F811
    """48 and 160 rows of a key head (prefix units of four and eight waves), own tokens in several ranges."""
    lens = ([1500, 3, 0, -1, 700, 129] + [64] * B)[:B]
    ask(Batch(nm, dtype, fmt, D, G * heads, heads, 64, 1500, lens))


@pytest.mark.parametrize("fmt,dtype", (("16", BF16), ("mx8", F16), ("mx4", BF16)))
@pytest.mark.parametrize("D,heads,G,P,lens", ((64, 1, 4, 0, [20000]), (64, 1, 2, 14000, [9000]), (64, 1, 4, 20000, [300, 0, -1]),
                                              (128, 4, 8, 2500, [1, 0] * 16)))
def test_more_parts_than_one_turn_joins(nm, dtype, fmt, D, heads, G, P, lens):  # noqa: F811
    """A row with more parts than the joining launch takes at a time: over 64 with 16 waves (few key heads), over 16
    with 4 (many row tiles)."""
    ask(Batch(nm, dtype, fmt, D, G * heads, heads, 256, P, lens))


def test_no_sequences(nm):  # noqa: F811
    """An empty batch gives an empty result, as rows of none do in the other calls; wrong arguments are refused all
    the same."""
    cache = nm.KVCache(4, 16, 2, 64, F16, "mx8")
    q, lens = torch.empty((0, 8, 64), dtype=F16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    table, pages = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((0, 3), (2,)))
    o = nm.attn_decode(q, cache, table, lens, prefix_pages=pages, prefix_len=20)
    assert o.shape == (0, 8, 64) and o.dtype == F16 and o.is_cuda
    out, lse = torch.empty_like(q), torch.empty((0, 8), device="cuda")
    ws = nm.attn_workspace(0, 8, cache, 48, 20)
    assert nm.attn_decode(q, cache, None, lens, out=out, lse=lse, ws=ws, stream=torch.cuda.Stream()) is out
    for bad in (lambda: nm.attn_decode(q[:, :7], cache, table, lens), lambda: nm.attn_decode(q, cache, table, lens, max_len=49),
                lambda: nm.attn_decode(q, cache, table, lens, out=torch.empty((0, 4, 64), dtype=F16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("fmt,dtype", (("16", F16), ("mx8", BF16), ("mx4", F16)))
@pytest.mark.parametrize("P", (0, 100))
def test_several_tokens_of_a_sequence(nm, fmt, dtype, P):  # noqa: F811
    """Several query tokens of a sequence at once (a draft, or a prompt's piece): a batch row each, with the sequence's
    pages and a length that ends at the token itself.  Each row sees what a row of its own batch would."""
    b = Batch(nm, dtype, fmt, 128, 8, 2, 16, P, [70, 1, 33])
    rows = torch.tensor([0, 0, 0, 0, 1, 2, 2], device="cuda")
    lens = torch.tensor([67, 68, 69, 70, 1, 32, 33], dtype=torch.int32, device="cuda")
    q = b.q[rows] + torch.arange(7, device="cuda").view(7, 1, 1).to(dtype) / 8
    o = nm.attn_decode(q, b.cache, b.table[rows], lens, prefix_pages=b.prefix_pages, prefix_len=P)
    for i, (r, n) in enumerate(zip(rows.tolist(), lens.tolist())):
        t = b.tokens(r)[:P + n]
        want, _, tol, _ = ref.attend(ref.f64(q[i]), b.qk[t], b.qv[t], 128 ** -0.5, dtype)
        assert (abs(ref.f64(o[i]) - want) <= tol).all(), i
