"""Plain 64-bit references (numpy, CPU) for the operators of include/nmserve.h,
written from the header's formulas; test infrastructure only."""
import numpy as np
import torch

from attn_reference import TINY, UNIT

F16 = torch.float16


def attend(q, k, v, seen, scale, dtype, one_operand):
    """q [rows][D], k and v [keys][D] of one key head in float64, seen [rows][keys].  Returns (o, lse, tolerance of o,
    tolerance of lse); only seen keys enter.

    Tolerance: a score's fp32 error is at most (D + 8) 2^-24 of sum |q k| scale plus 2^-22 of its size for the base-2
    factor and the exponential; it moves a weight by that much, relative, and the sum that divides it likewise.  With
    one operand each weight is rounded once to dtype (half a step u), in the sum that divides, too: o moves by at most
    2 u / (1 - u) of the weighted mean of |v|.  With two operands 2^-16 (bfloat16) or 2^-22 of a weight is lost.  In fp16
    weights lose at most 2^-32 of the row's largest one besides (both in the sum and in the divisor).  fp32 sums over the
    keys add (keys + 32) 2^-24 each.  Then one rounding of o.  lse adds up the weights before their rounding."""
    rows, D = q.shape
    o, lse = np.zeros((rows, D)), np.full(rows, -np.inf)
    tol, ltol = np.full((rows, D), TINY[dtype]), np.zeros(rows)
    u = UNIT[dtype]
    lost = 2 * u / (1 - u) if one_operand else 2 * (2.0 ** -22 if dtype == F16 else 2.0 ** -16)
    floor = 2.0 ** -32 if dtype == F16 else 0.0
    for r in range(rows):
        kk, vv = k[seen[r]], v[seen[r]]
        n = len(kk)
        if n == 0:
            continue
        s = kk @ q[r] * scale
        p = np.exp(s - s.max())
        l = p.sum()
        o[r] = p / l @ vv
        lse[r] = s.max() + np.log(l)
        size = (np.abs(kk) @ np.abs(q[r]) * abs(scale)).max()
        err = 2 * ((D + 8) * 2.0 ** -24 * size + 2.0 ** -22 * np.abs(s).max() + 2.0 ** -22)
        mean = p / l @ np.abs(vv)
        t = (2 * err + lost + 2 * (n + 32) * 2.0 ** -24) * mean + floor * (np.abs(vv).sum(0) + n * mean) / l
        tol[r] = t + u * (np.abs(o[r]) + t) + TINY[dtype]
        ltol[r] = err + (n + 32) * 2.0 ** -24 + 2.0 ** -22 * (1 + abs(lse[r]))
    return o, lse, tol, ltol


def prompt(q, k, v, starts, k_starts, scale, dtype):
    """attn_prompt of float64 arrays; rows of no sequence are NaN.  Returns (o, lse, tolerances)."""
    T, hq, D = q.shape
    G = hq // k.shape[1]
    o, lse = np.full((T, hq, D), np.nan), np.full((T, hq), np.nan)
    tol, ltol = np.zeros((T, hq, D)), np.zeros((T, hq))
    for a, z, ka, kz in zip(starts, starts[1:], k_starts, k_starts[1:]):
        nq, nk = z - a, kz - ka
        seen = np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq
        for h in range(hq):
            o[a:z, h], lse[a:z, h], tol[a:z, h], ltol[a:z, h] = attend(
                q[a:z, h], k[ka:kz, h // G], v[ka:kz, h // G], seen, scale, dtype, True)
    return o, lse, tol, ltol


def close(got, want, tol, what):
    """Every element of got (float64) within tol of want; NaN where want is NaN, infinities equal."""
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), what
    with np.errstate(invalid="ignore"):
        over = np.abs(got[fine] - want[fine]) / tol[fine]
    assert len(over) == 0 or np.nanmax(over) <= 1 and not np.isnan(over).any(), \
        (what, int((~(over <= 1)).sum()), float(np.nanmax(over)))


def plan(table, lens, free, n_free, page, adds, rows):
    """One step of the book in plain Python; lists are changed in place.  Returns (n_free, starts, slots, positions,
    granted)."""
    B, width, capacity = len(lens), len(table[0]), len(free)
    pages = lambda n: -(-n // page)                                                                       # noqa: E731
    n_free = min(max(n_free, 0), capacity)
    granted, given = [0] * B, []
    for b in range(B):
        if lens[b] > 0 and adds[b] < 0:
            keep = max(lens[b] + adds[b], 0)
            granted[b] = keep - lens[b]
            given += table[b][min(pages(keep), width):min(pages(lens[b]), width)]
    for i, p in enumerate(reversed(given)):
        if n_free + i < capacity:
            free[n_free + i] = p
    n_free = min(n_free + len(given), capacity)
    starts, slots, positions, closed = [0], [], [], False
    for b in range(B):
        if lens[b] >= 0 and adds[b] > 0 and lens[b] + adds[b] < 2 ** 31 and pages(lens[b] + adds[b]) <= width:
            new = pages(lens[b] + adds[b]) - min(pages(lens[b]), width)
            closed = closed or new > n_free or len(slots) + adds[b] > rows
            if not closed:
                granted[b] = adds[b]
                for i in range(new):
                    n_free -= 1
                    table[b][pages(lens[b]) + i] = free[n_free]
                for t in range(lens[b], lens[b] + adds[b]):
                    p = table[b][t // page]
                    slots.append(-1 if p < 0 else p * page + t % page)
                    positions.append(t)
        starts.append(len(slots))
    for b in range(B):
        lens[b] += granted[b]
    slots += [-1] * (rows - len(slots))
    positions += [0] * (rows - len(positions))
    return n_free, starts, slots, positions, granted
