"""nm_attn_decode against its formula where the scores are free of rounding: what is left is the exponential, the
weights, the sums and one rounding of o, so that a weight held in 16 bits alone would show."""
import numpy as np
import pytest
import torch

import attn_reference as ref
from test_gpu_attn import BF16, F16, FORMATS, Batch, nm, rnd  # noqa: F401  (nm: the fixture)

pytestmark = pytest.mark.gpu

MX4 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def grid(shape, dtype, *tag):
    """Values that every format holds exactly: e2m1's, a 6 in each block of 32 columns."""
    code = (rnd(shape, torch.float32, *tag).cpu().abs() * 3.5).long().clamp(max=7)
    x = MX4[code] * torch.sign(rnd(shape, torch.float32, "sign", *tag).cpu())
    x[..., ::32] = 6.0
    return x.to(dtype).cuda()


def refill(b, k, v):
    """Other keys and values into a Batch's slots."""
    b.k, b.v = k, v
    b.nm.kv_write(b.cache, k, v, b.slots.cuda())
    b.qk, b.qv = (ref.quantised(ref.f64(t), b.fmt, b.dtype) for t in (k, v))


def attend_exact(q, keys, values, scale, dtype, small):
    """(o, tolerance) of one sequence whose q . k have no rounding in fp32 (few bits each, sums far below 2^24 steps).

    Tolerance of a weight, relative: the base-2 factor, the product with it and the difference from the reference are
    three roundings of at most 2^-23 of the largest score (base 2, so 1.5 |s|) each and the exponential adds 2^-22; the
    16-bit pair that carries it into the product leaves half a step of half a step, UNIT^2.  `small`: what a weight may
    lose beside that, as a share of the largest one (fp16's subnormals).  fp32 sums over the tokens and the joins:
    (tokens + 32) 2^-24 of the magnitudes.  Numerator and denominator both, then one rounding of o."""
    n, heads, D = keys.shape
    G = q.shape[0] // heads
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(q.shape[0]):
        k, v = keys[:, h // G], values[:, h // G]
        s = k @ q[h] * scale
        p = np.exp(s - s.max())
        w = p / p.sum()
        o[h] = w @ v
        weight = 3 * 2.0 ** -23 * 1.5 * np.abs(s).max() + 2.0 ** -22 + ref.UNIT[dtype] ** 2
        t = 2 * (weight + (n + 32) * 2.0 ** -24) * (w @ np.abs(v)) + small * np.abs(v).sum(0) / p.sum()
        tol[h] = t + ref.UNIT[dtype] * (np.abs(o[h]) + t) + ref.TINY[dtype]
    return o, tol


# A weight's two fp16 parts end at multiples of 2^-24 and the largest weight is at least 2^7; bfloat16 reaches 2^-126.
SMALL = {F16: 2.0 ** -32, BF16: 0.0}


def check(b, scale, small):
    """`small`: see attend_exact()."""
    o = b.run(scale=scale)
    for i, n in enumerate(b.lens):
        t = b.tokens(i)
        if t:
            want, tol = attend_exact(ref.f64(b.q[i]), b.qk[t], b.qv[t], scale, b.dtype, small)
            err = np.abs(ref.f64(o[i]) - want)
            assert (err <= tol).all(), (i, n, float((err / tol).max()))


# Own tokens in one range and in several; a prefix with up to 16, 17 to 32, 33 to 128 and more rows of a key head.
SHAPES = ((4, 2, 0, [64, 1, 33]), (8, 1, 0, [40, 600]), (4, 4, 70, [5, 30]), (4, 1, 90, [9, 0, 20, 3, 1]),
          (16, 2, 100, [3, 11, 0, 7, 20]), (8, 1, 64, [5] * 20), (16, 1, 200, [10, 0, 33] * 6))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("D", (64, 128, 256))
@pytest.mark.parametrize("hq,heads,P,lens", SHAPES)
def test_weights_keep_their_bits(nm, dtype, fmt, D, hq, heads, P, lens):  # noqa: F811
    b = Batch(nm, dtype, fmt, D, hq, heads, 16, P, lens)
    b.q = rnd(b.q.shape, torch.float32, "eq", D).round().clamp(-1, 1).to(dtype)
    refill(b, grid(b.k.shape, dtype, "ek", D), grid(b.v.shape, dtype, "ev", D))
    assert np.array_equal(b.qk, ref.f64(b.k)) and np.array_equal(b.qv, ref.f64(b.v))
    check(b, 0.5 / np.sqrt(D), SMALL[dtype])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", (F16, BF16))
@pytest.mark.parametrize("gap", (16.7, 17.5, 19.0))
@pytest.mark.parametrize("D,hq,heads,P,lens", ((128, 4, 2, 0, [32, 33]), (64, 4, 1, 0, [700]), (128, 4, 4, 200, [3]),
                                               (128, 4, 1, 90, [1, 0, 2, 3, 1]), (64, 8, 1, 300, [5] * 20),
                                               (128, 16, 1, 300, [2, 0] * 9), (256, 32, 4, 150, [1] * 6)))
def test_far_tokens_count(nm, dtype, fmt, gap, D, hq, heads, P, lens):  # noqa: F811
    """One token far above all others, with values of zero (a first token that takes most of the weight): what o is
    comes from the others, each of them below fp16's least number beside that token's weight of one."""
    b = Batch(nm, dtype, fmt, D, hq, heads, 16, P, lens)
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = 1.0
    k = torch.zeros_like(b.k)
    k[0, :, 0] = 6.0
    v = grid(b.v.shape, dtype, "fv", D) * 4096
    v[0] = 0.0
    refill(b, k, v)
    check(b, gap / 6, SMALL[dtype])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", (2.0 ** 121, 2.0 ** -118))
@pytest.mark.parametrize("hq,heads,P,lens", ((4, 2, 0, [90, 33]), (4, 1, 0, [900]), (4, 1, 90, [40, 0, 2, 3, 1]),
                                             (8, 1, 300, [5] * 20)))
def test_bfloat16_values_near_the_ends(nm, fmt, size, hq, heads, P, lens):  # noqa: F811
    """Values up to 6 2^121 with scores that climb from 0 over 0.9 to 7 (base 2) in the last tokens: weights above one
    would take the sums past fp32, weights of at most one, 2^-8 for the first tokens, keep them below 2^127.  And
    values down to the type's least normal ones."""
    b = Batch(nm, BF16, fmt, 128, hq, heads, 16, P, lens)
    b.q = torch.zeros_like(b.q)
    b.q[..., 0] = 1.0
    k = torch.zeros_like(b.k)
    k[..., 0] = 0.5                                   # (a value of every format)
    for i in range(len(lens)):
        t = b.tokens(i)
        k[t[:16], :, 0] = 0.0
        if len(t) > 32:
            k[t[-2:], :, 0] = 4.0
    refill(b, k, (grid(b.v.shape, BF16, "bv").float() * size).to(BF16))
    check(b, 7 * np.log(2) / 4, SMALL[BF16])
