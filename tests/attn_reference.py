"""Plain 64-bit references (numpy, CPU) for the operators of include/nmattn.h,
written from the header's formulas; test infrastructure only.

16-bit tensors are handled as their values in float64; quantised blocks through
a table of the format's values and its midpoints."""
import numpy as np
import torch

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}      # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}    # half a step of the subnormals
LARGEST = {torch.float16: 65504.0, torch.bfloat16: float(torch.finfo(torch.bfloat16).max)}


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- quantised blocks -------------------------------------------------------

def _e4m3():
    v = []
    for code in range(127):                                        # 127 is the format's NaN
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


GRID = {"mx8": _e4m3(), "mx4": np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])}
TOP = {"mx8": 448.0, "mx4": 6.0}


LEAST = {(torch.bfloat16, "mx8"): -126, (torch.bfloat16, "mx4"): -126,       # least exponent of a scale
         (torch.float16, "mx8"): -14, (torch.float16, "mx4"): -22}


def quantised(x, fmt, dtype, read=False):
    """The values a cache of format fmt holds for x [..., D] of dtype; with
    read, as they are read back into it (saturating)."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "16":
        return x
    blocks = x.reshape(-1, 32)
    out = np.empty_like(blocks)
    grid, mid = GRID[fmt], (GRID[fmt][1:] + GRID[fmt][:-1]) / 2
    for i, b in enumerate(blocks):
        if not np.isfinite(b).all():
            out[i] = np.nan
            continue
        top, e = np.abs(b).max(), LEAST[dtype, fmt]
        while top > TOP[fmt] * 2.0 ** e:
            e += 1
        a = np.abs(b) * 2.0 ** -e
        below, upto = np.searchsorted(mid, a, side="left"), np.searchsorted(mid, a, side="right")
        code = np.where(below % 2 == 0, below, upto)
        out[i] = np.copysign(grid[code] * 2.0 ** e, b)
    out = out.reshape(x.shape)
    return out if not read else np.clip(out, -LARGEST[dtype], LARGEST[dtype])


# ---- norm and rotation --------------------------------------------------------

def qk(x, w, eps, positions, inv_freq, interleaved):
    """(y, magnitude): the result and |n_a| + |n_b| of each column's pair."""
    x = f64(x)
    D, rot = x.shape[-1], 2 * len(inv_freq)
    n = x
    if w is not None:
        n = x / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps) * f64(w)
    angle = f64(positions)[:, None, None] * f64(inv_freq)[None, None, :]
    c, s = np.cos(angle), np.sin(angle)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, mag = n.copy(), np.abs(n)
    y[..., a] = n[..., a] * c - n[..., b] * s
    y[..., b] = n[..., b] * c + n[..., a] * s
    mag[..., a] = mag[..., b] = np.abs(n[..., a]) + np.abs(n[..., b])
    return y, mag


def qk_close(got, x, w, eps, positions, inv_freq, interleaved):
    """fp32 evaluation: D squares summed (D 2^-24), root, quotient and weight (8 units), the pair's products and
    their sum (3 units), sine and cosine of an fp32 argument up to pi (2^-22 absolute), then one rounding."""
    y, mag = qk(x, w, eps, positions, inv_freq, interleaved)
    D = y.shape[-1]
    tol = mag * ((D + 16) * 2.0 ** -24 + 2.0 ** -21)
    tol = tol + UNIT[x.dtype] * (np.abs(y) + tol) + TINY[x.dtype]
    bad = np.abs(f64(got) - y) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(f64(got) - y) / tol).max()))


# ---- attention ------------------------------------------------------------------

def attend(q, keys, values, scale, dtype):
    """One sequence: q [Hq][D], keys and values [tokens][heads][D] (the cache's
    values, float64).  Returns (o, lse, tolerance of o, tolerance of lse).

    Tolerance: a score's fp32 error is at most (D + 8) 2^-24 of sum |q k| scale
    plus 2^-22 of its size for the
    base-2 factor and the exponential; it moves a weight by that much,
    relative.  Each weight is rounded once to dtype (half a step); weights below
    fp16's normal range lose at most 2^-25 of the largest one, each.  fp32 sums
    over the tokens add (tokens + 32) 2^-24.  Then one rounding of o."""
    Hq, D = q.shape
    n, heads, _ = keys.shape
    G = Hq // heads
    o, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    tol, ltol = np.full((Hq, D), TINY[dtype]), np.zeros(Hq)
    if n == 0:
        return o, lse, tol, ltol
    unit = UNIT[dtype]
    for h in range(Hq):
        k, v = keys[:, h // G], values[:, h // G]
        s = k @ q[h] * scale
        p = np.exp(s - s.max())
        l = p.sum()
        w = p / l
        o[h] = w @ v
        lse[h] = s.max() + np.log(l)
        size = np.abs(k) @ np.abs(q[h]) * abs(scale)
        err = 2 * ((D + 8) * 2.0 ** -24 * size.max() + 2.0 ** -22 * np.abs(s).max() + 2.0 ** -22)
        rel = 2 * err + unit + (n + 32) * 2.0 ** -24
        floor = 2.0 ** -25 if dtype == torch.float16 else 0.0
        t = rel * (w @ np.abs(v)) + floor * np.abs(v).sum(0) / l
        tol[h] = t + UNIT[dtype] * (np.abs(o[h]) + t) + TINY[dtype]
        ltol[h] = err + (n + 32) * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(lse[h]))
    return o, lse, tol, ltol
