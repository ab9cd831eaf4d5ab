"""Attention of prompts and trees where a wrong token would stand out: long prompts in fp16, values in one tile of keys only,
and infinities and NaN in quantised caches (where one marks its block of 32 columns) that a draft does not see."""
import math
import random

import numpy as np
import pytest
import torch

import attn_reference as ref
import serve_reference as sref
from test_gpu_prompt import check, rnd, starts_of
from test_gpu_tree import Case, nm, tree  # noqa: F401

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("pieces", [[(1, 5000)], [(40, 3001), (7, 20), (0, 900), (3, 2)], [(130, 4097)]])
def test_few_rows_behind_many_keys_in_fp16(nm, pieces):  # noqa: F811
    nq, nk = zip(*pieces)
    q, k, v = (rnd((n, h, 128), F16, "few", n, i) for i, (n, h) in enumerate(((sum(nq), 4), (sum(nk), 1), (sum(nk), 1))))
    check(nm, q, k, v, starts_of(nq), starts_of(nk))


def rows_against_formula(q, k, v, out, rows, nq, nk):
    for i in rows:
        n = i + 1 + nk - nq
        o, _, tol, _ = sref.prompt(ref.f64(q[i:i + 1]), ref.f64(k[:n]), ref.f64(v[:n]), [0, 1], [0, n], q.shape[-1] ** -0.5,
                                   q.dtype)
        sref.close(ref.f64(out[i:i + 1]), o, tol, i)


@pytest.mark.parametrize("D", (64, 128, 256))
def test_long_prompt_rows_in_fp16(nm, D):  # noqa: F811
    n = 4100
    q, k, v = (rnd((n, h, D), F16, "long", i) for i, h in enumerate((4, 1, 1)))
    out = nm.attn_prompt(q, k, v, starts_of([n]))
    rows_against_formula(q, k, v, out, (0, 63, 64, 1000, 2047, 4098, 4099), n, n)


@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D", (64, 128, 256))
@pytest.mark.parametrize("nq", (4100, 20))
def test_values_in_one_step_of_keys(nm, dtype, D, nq):  # noqa: F811
    """All values are zero but those of 32 keys: what the rows behind them get is these keys' weights, in whole prompts and
    in ranges of keys."""
    nk = 4100
    q, k = rnd((nq, 4, D), dtype, "one", 0), rnd((nk, 1, D), dtype, "one", 1)
    some = rnd((nk, 1, D), dtype, "one", 2)
    for step in (0, 1, 2, 3, 64, 65, 127, 128):
        v = torch.zeros_like(some)
        at = slice(32 * step, min(32 * step + 32, nk))
        v[at] = some[at]
        out = nm.attn_prompt(q, k, v, starts_of([nq]), starts_of([nk]))
        before = nk - nq                                                # keys that the first row sees besides its own
        rows = {0, nq // 2, nq - 1, *(min(max(at.start + d - before, 0), nq - 1) for d in (-1, 0, 1, 30, 31, 32, 64))}
        rows_against_formula(q, k, v, out, sorted(rows), nq, nk)


def unseen(nm, c, odd):  # noqa: F811
    """Drafts whose values, then keys too, hold `odd` in one column: rows that do not see them as before, rows that do
    without a finite value in its block of columns.

    A row that does not see the draft has the same weights and the same divisor; its sum of two terms a token (the weight's two
    operands) may be added in another order, which moves it by 2 (2 n) 2^-24 max |v| at most; then both are rounded, half a
    step each."""
    n, N, D, u = c.lens[0], c.N, c.D, ref.UNIT[c.dtype]
    clean = c.run()
    top = max(np.abs(v).max() for v in c.v)
    moved = 4 * n * 2.0 ** -24 * top
    bad = rnd((1, c.heads, D), c.dtype, "bad")
    bad[0, 0, 37] = odd
    block = slice(32, 64)
    for j in (0, N // 2, N - 1):
        for b in range(len(c.lens)):
            at = c.slots[b][n - N + j:n - N + j + 1]
            k, v = nm.kv_read(c.cache, at)
            nm.kv_write(c.cache, k, bad, at)
            values = c.run()
            nm.kv_write(c.cache, torch.full_like(bad, odd), bad, at)
            both = c.run()
            nm.kv_write(c.cache, k, v, at)                              # read back and written again: the same codes
            for i in range(N):
                if c.masks[b][i] >> j & 1:
                    assert not values[b, i, :, block].isfinite().any() and not both[b, i].isfinite().any()
                    assert values[b, i, :, :32].isfinite().all() and values[b, i, :, 64:].isfinite().all()
                    continue
                want = clean[b, i].double()
                for got in (values, both):
                    d = (got[b, i].double() - want).abs()
                    assert (d <= moved + u * (2 * want.abs() + moved) + 2 * ref.TINY[c.dtype]).all(), (j, b, i)
            other = [x for x in range(len(c.lens)) if x != b]
            assert torch.equal(values[other], clean[other]) and torch.equal(both[other], clean[other])
    assert torch.equal(c.run(), clean)


@pytest.mark.parametrize("fmt", ("mx8", "mx4"))
@pytest.mark.parametrize("odd", (math.nan, math.inf))
@pytest.mark.parametrize("dtype,D,G,N", [(F16, 64, 1, 6), (BF16, 128, 4, 6), (F16, 128, 8, 12), (BF16, 64, 8, 40),
                                         (F16, 256, 2, 6), (BF16, 256, 4, 12)])
def test_unseen_in_quantised_caches(nm, fmt, dtype, D, G, N, odd):  # noqa: F811
    masks = [[1 << i for i in range(N)], tree(N, random.Random(3))]
    unseen(nm, Case(nm, fmt, dtype, D, 1, G, N, [150, 150], 64, masks=masks), odd)


@pytest.mark.parametrize("fmt", ("mx8", "mx4"))
@pytest.mark.parametrize("odd", (math.nan, math.inf))
@pytest.mark.parametrize("dtype,D,G,N", [(BF16, 128, 4, 12), (F16, 64, 8, 20), (F16, 128, 4, 33)])
def test_unseen_in_quantised_caches_shared_form(nm, fmt, dtype, D, G, N, odd):  # noqa: F811
    masks = [[1 << i for i in range(N)], tree(N, random.Random(3))]
    unseen(nm, Case(nm, fmt, dtype, D, 1, G, N, [150, 150], 64, masks=masks).widen(), odd)
