"""Float64 CPU oracle of the generation operators: the 8-bit product and the sampler.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (same rules as ``oracle/dense_kl.py``).

    quantise   s = max_k |x_k| * fl(1/127) in float32,  q_k = rint(x_k / s) in [-127, 127]
    product    y = (q w^T) * s * t
    sample     z = (x - m) * fl(1/T) in float32, w = floor(2^40 exp(z)), filters, draw

The quantised values are float32 arithmetic by definition, so they are computed in it; the
product and the exponentials are float64.
"""
from __future__ import annotations

import numpy as np

ONE = 2.0 ** 40


def quantize_int8(x):
    """(q int8 [M, K], scale float32 [M]) of float32 values x [M, K]."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(axis=1)
    with np.errstate(invalid="ignore"):
        scale = (amax * (np.float32(1) / np.float32(127))).astype(np.float32)
        scale[~np.isfinite(x).all(axis=1)] = np.nan
    q = np.zeros(x.shape, dtype=np.int8)
    for m in range(x.shape[0]):
        if scale[m] > 0:
            q[m] = np.clip(np.rint(x[m] / scale[m]), -127, 127).astype(np.int8)
    return q, scale


def int8_matmul(xq, x_scale, wq, w_scale):
    """float64 [M, N]."""
    s = np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T
    return s * np.asarray(x_scale, dtype=np.float64)[:, None] * np.asarray(w_scale, dtype=np.float64)[None, :]


def ranked(row):
    """Ids that can be drawn, by logit descending, ties by the lower id."""
    row = np.asarray(row, dtype=np.float32)
    ids = np.flatnonzero(row > -np.inf)  # NaN compares false
    return ids[np.lexsort((ids, -row[ids].astype(np.float64)))]


def sample_weights(row, temperature):
    """(z float32 [V], weights float64 [V], whole numbers) of one row."""
    row = np.where(np.isnan(np.asarray(row, dtype=np.float32)), -np.inf, row).astype(np.float32)
    m = row.max()
    t = np.float32(temperature)
    inv = np.float32(1) / t if t > 0 else np.float32(1)
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(row == m, np.float32(0), (row - m) * inv).astype(np.float32)
        w = np.floor(ONE * np.exp(z.astype(np.float64)))
    return z, np.where(row > -np.inf, np.nan_to_num(w), 0.0)


def kept_ids(row, temperature, top_k, top_p, min_p, tol=0.0):
    """(surely, possibly): boolean [V], the ids the filters keep whatever the exponentials'
    rounding (relative tol), and those they may keep."""
    row = np.asarray(row, dtype=np.float32)
    order = ranked(row)
    z, w = sample_weights(row, temperature)
    k = 1 if not np.float32(temperature) > 0 else int(top_k)
    if k > 0:
        order = order[:k]
    sure, may = np.zeros(row.size, bool), np.zeros(row.size, bool)
    ws = w[order]
    before = np.concatenate([[0.0], np.cumsum(ws)[:-1]])
    total = ws.sum()
    p = float(np.float32(top_p))
    first = np.arange(order.size) == 0
    top = row[order] == row[order[0]] if order.size else first
    e = np.exp(z[order].astype(np.float64))
    mp = float(np.float32(min_p))
    for mark, sign in ((sure, -1.0), (may, 1.0)):
        keep = first | (p >= 1) | (before < p * total + sign * tol * total)
        keep &= top | (e >= mp * (1 - sign * tol))
        mark[order] = keep
    return sure, may


def sample_row(row, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tol=2.0 ** -20):
    """Tokens that the definition allows for one row when exponentials are off by a relative
    tol / 4 at most, as {token: (lowest, highest) log-probability}: the ids that may be kept
    between the earliest and the latest that the draw can reach.  {-1: (nan, nan)} when nothing
    can be drawn."""
    row = np.asarray(row, dtype=np.float32)
    if ranked(row).size == 0:
        return {-1: (float("nan"), float("nan"))}
    z, w = sample_weights(row, temperature)
    sets = kept_ids(row, temperature, top_k, top_p, min_p, tol)
    totals, drawn = [], []
    for keep in sets:
        c = np.cumsum(np.where(keep, w, 0.0))
        totals.append(c[-1])
        for shift in (-tol, 0.0, tol):
            r = min(max(np.floor((float(np.float32(u)) + shift) * c[-1]), 0.0), c[-1] - 1)
            drawn.append(int(np.flatnonzero(c > r)[0]))
    ids = np.arange(min(drawn), max(drawn) + 1)
    ids = ids[sets[1][ids] & (w[ids] > 0)]
    lo, hi = np.log(max(totals) / ONE), np.log(min(totals) / ONE)
    return {int(t): (float(z[t]) - lo, float(z[t]) - hi) for t in ids}
