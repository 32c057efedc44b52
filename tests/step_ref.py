"""The operators between a verify step's products, evaluated in 64 bits with
numpy from their definitions (imported by test modules only)."""
import math

import numpy as np


def turns(rot, base=10000.0):
    return np.array([base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)])


def rotate(x, pos, t, off, layout, mscale=1.0):
    """(rotated x, |a| + |b| of each value's pair, 0 where copied), in fp64."""
    x = np.asarray(x, dtype=np.float64)
    out, size = x.copy(), np.zeros_like(x)
    half = len(t)
    for i in range(half):
        ia, ib = (off + i, off + i + half) if layout == "half" else (off + 2 * i, off + 2 * i + 1)
        part = pos.astype(np.float64) * t[i]
        r = (2 * math.pi * (part - np.round(part)))[:, None]
        a, b = x[..., ia], x[..., ib]
        out[..., ia] = mscale * (a * np.cos(r) - b * np.sin(r))
        out[..., ib] = mscale * (a * np.sin(r) + b * np.cos(r))
        size[..., ia] = size[..., ib] = abs(mscale) * (np.abs(a) + np.abs(b))
    return out, size


def attention(q, kc, vc, table, ctx, start, mask, scale):
    """out, lse and, per row, what the tolerances need: the weighted |v| and
    the largest sum |q k| * scale of a seen key."""
    q, kc, vc = (np.asarray(x, dtype=np.float64) for x in (q, kc, vc))
    total, heads, dim = q.shape
    page, kv = kc.shape[1], kc.shape[2]
    out, lse = np.zeros(q.shape), np.full((total, heads), -np.inf)
    absv, big = np.zeros(q.shape), np.zeros((total, heads))
    for s in range(len(ctx)):
        n = start[s + 1] - start[s]
        where = np.arange(ctx[s] + n)
        slot = table[s][where // page].astype(np.int64), where % page
        k, v = kc[slot], vc[slot]  # (len, kv, dim)
        for i in range(n):
            row = start[s] + i
            seen = np.array([p < ctx[s] or bool(int(mask[row]) >> int(p - ctx[s]) & 1) for p in where], dtype=bool)
            if not seen.any():
                continue
            for g in range(kv):
                h = slice(g * (heads // kv), (g + 1) * (heads // kv))
                kk, vv = k[seen, g], v[seen, g]
                x = q[row, h] @ kk.T * scale
                top = x.max(1, keepdims=True)
                w = np.exp(x - top)
                z = w.sum(1, keepdims=True)
                out[row, h], absv[row, h] = w / z @ vv, w / z @ np.abs(vv)
                lse[row, h] = (top + np.log(z))[:, 0]
                big[row, h] = (np.abs(q[row, h]) @ np.abs(kk).T).max(1) * abs(scale)
    return out, lse, absv, big


def sample(row, t, k, p, least, u):
    """(id, probability, margin): margin is how near, relative to the kept
    mass, the choice came to another one."""
    row = np.asarray(row, dtype=np.float64) + 0.0
    live = np.isfinite(row) if not np.isposinf(row).any() else np.isposinf(row)
    live &= ~np.isnan(row)
    idx = np.flatnonzero(live)
    if not idx.size:
        return -1, 0.0, 1.0
    x = row[idx]
    order = np.lexsort((idx, -x))
    if not t > 0:
        return int(idx[order[0]]), 1.0, 1.0
    x = x[order]
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(x == x[0], 0.0, (x - x[0]) / t))
    margin = 1.0
    keep = order.size if k <= 0 else min(k, order.size)
    w, order = w[:keep], order[:keep]
    if p < 1:
        sums = np.cumsum(w)
        goal = max(p, 0.0) * sums[-1]
        before = sums - w
        keep = max(1, int(np.sum(before < goal)))
        exact = np.all(w == np.floor(w))  # all weights equal to 1 or 0: no rounding on either side
        if not exact:
            margin = min(margin, np.abs(before[1:] - goal).min(initial=1.0) / sums[-1])
        w, order = w[:keep], order[:keep]
    if least > 0:
        good = w >= least
        good[0] = True
        if not np.all(w == np.floor(w)):
            # a weight is held within 2^-39 of itself and 2^-46: twice that is a margin of 2^-30
            margin = min(margin, (np.abs(w[1:] - least) / (least * 2.0 ** -39 + 2.0 ** -46)).min(initial=1e9) * 2.0 ** -31)
        w, order = w[good], order[good]
    by = np.argsort(idx[order])
    sums = np.cumsum(w[by])
    at = min(int(np.searchsorted(sums, u * sums[-1], side="right")), len(by) - 1)
    if not np.all(w == np.floor(w)):
        margin = min(margin, np.abs(sums[:-1] - u * sums[-1]).min(initial=1.0) / sums[-1])
    j = by[at]
    return int(idx[order[j]]), float(w[j] / sums[-1]), margin
