"""What follows a verify step's logits, evaluated in 64 bits with numpy from the
definitions (imported by test modules only)."""
import numpy as np


def probs(row, t, k, p, least):
    """(distribution, margin): margin is how near, relative to the kept mass, a
    cut came to falling elsewhere."""
    row = np.asarray(row, dtype=np.float64) + 0.0
    out = np.zeros(row.size)
    live = np.isposinf(row) if np.isposinf(row).any() else np.isfinite(row)
    idx = np.flatnonzero(live)
    if not idx.size:
        return out, 1.0
    x = row[idx]
    order = np.lexsort((idx, -x))
    if not t > 0:
        out[idx[order[0]]] = 1.0
        return out, 1.0
    x = x[order]
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(x == x[0], 0.0, (x - x[0]) / t))
    margin = 1.0
    if 0 < k < order.size:
        w, order = w[:k], order[:k]
    if p < 1:
        sums = np.cumsum(w)
        before, goal = sums - w, max(p, 0.0) * sums[-1]
        keep = max(1, int(np.sum(before < goal)))
        margin = min(margin, np.abs(before[1:] - goal).min(initial=1.0) / sums[-1])
        w, order = w[:keep], order[:keep]
    if least > 0:
        good = w >= least
        good[0] = True
        margin = min(margin, np.abs(w[1:] / least - 1).min(initial=1.0))
        w, order = w[good], order[good]
    out[idx[order]] = w / w.sum()
    return out, margin


def verify(p, q, tokens, parent, u, u_next):
    """One sequence: p, q (nodes, V) in 64 bits (q None: chosen drafts).  (path,
    next, margin): how near, relative to their terms, a decision came to another."""
    p = np.where(np.isnan(p), 0.0, np.asarray(p, dtype=np.float64))
    V, at, path, margin = p.shape[1], 0, [0], 1.0
    while True:
        c, left, into, gone = 0.0, 1.0, None, set()
        for i in range(at + 1, len(tokens)):
            if parent[i] != at:
                continue
            x = int(tokens[i])
            inside = 0 <= x < V
            if q is None:
                here, rest = 1.0, p[at, x] if inside and x not in gone else 0.0
            else:
                here = q[at, x] if inside else 0.0
                rest = p[at, x] - c * here if inside else 0.0
            a = float(u[i]) * here * left
            size = a + (p[at, x] if inside else 0.0) + c * here
            if size > 0:
                margin = min(margin, abs(a - rest) / size)
            if a < rest:
                into = i
                break
            if q is None:
                if rest > 0:
                    gone.add(x)
                    left -= rest
            elif left > 0:
                c += left
                left = np.maximum(p[at] - c * q[at], 0.0).sum()
        if into is None:
            break
        at = into
        path.append(at)
    r = np.maximum(p[at], 0.0) if q is None else np.maximum(p[at] - c * np.nan_to_num(q[at]), 0.0)
    r[list(gone)] = 0.0
    if not r.sum() > 0:
        r = np.maximum(p[at], 0.0)
    sums = np.cumsum(r)
    if not sums[-1] > 0:
        return path, -1, margin
    goal = float(u_next) * sums[-1]
    nxt = int(np.flatnonzero(sums > goal)[0])
    return path, nxt, min(margin, np.abs(sums[r > 0] - goal).min() / sums[-1])


def outcome(p, q, k):
    """The distribution of the token that comes out where k drafts drawn from q
    are tried at one node against p, by summing over all draws; of chosen drafts,
    q is the list of them."""
    V, out = p.size, np.zeros(p.size)
    if not isinstance(q, np.ndarray):
        r, left, reach = p.copy(), 1.0, 1.0
        for x in q:
            take = min(1.0, r[x] / left) if left > 0 else 0.0
            out[x] += reach * take
            reach *= 1 - take
            left -= r[x]
            r[x] = 0.0
        return out + (reach * r / r.sum() if r.sum() > 0 else 0.0)
    c, left, reach = 0.0, 1.0, 1.0
    for _ in range(k):
        rest = np.maximum(p - c * q, 0.0)
        take = np.minimum(1.0, np.divide(rest, q * left, out=np.full(V, 1.0), where=q * left > 0))
        out += reach * q * take
        reach *= 1 - (q * take).sum()
        c += left
        left = np.maximum(p - c * q, 0.0).sum()
        if left <= 1e-300:
            break
    rest = np.maximum(p - c * q, 0.0)
    return out + (reach * rest / rest.sum() if rest.sum() > 0 else reach * p)


def commit(kc, vc, table, ctx, path, count):
    """kc, vc (layers, pages, page, kv, dim) after the moves, on copies."""
    kc, vc = kc.copy(), vc.copy()
    page = kc.shape[2]
    for s in range(len(ctx)):
        old_k, old_v = kc.copy(), vc.copy()  # all moves read what was there before any
        for i in range(count[s]):
            a, b = ctx[s] + int(path[s][i]), ctx[s] + i
            kc[:, table[s][b // page], b % page] = old_k[:, table[s][a // page], a % page]
            vc[:, table[s][b // page], b % page] = old_v[:, table[s][a // page], a % page]
    return kc, vc


_E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)][:127])


def e4m3(x):
    """Each x as the nearest e4m3 number, of two as near the one whose last bit is 0; NaN for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.searchsorted(_E4M3, a).clip(1, 126)
    lo = hi - 1
    down, up = a - _E4M3[lo], _E4M3[hi] - a
    pick = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(x), np.copysign(_E4M3[pick], x), np.nan)


def quantize(x, block):
    """x (pages, page, kv, dim): its e4m3 numbers and (pages, page / block, kv) scales."""
    x = np.asarray(x, dtype=np.float64)
    pages, page, kv, dim = x.shape
    y = x.reshape(pages, page // block, block, kv, dim)
    most = np.where(np.isfinite(y), np.abs(y), 0.0).max(axis=(2, 4))
    e = np.zeros(most.shape)
    for i, m in np.ndenumerate(most):
        if m > 0:
            k = -80
            while k < 120 and 448.0 * 2.0 ** k < m:
                k += 1
            e[i] = k
    scale = 2.0 ** e
    return e4m3(y / scale[:, :, None, :, None]).reshape(x.shape), scale


def attention(q, seqs, scale):
    """q (rows, heads, dim); seqs: (first row, keys (len, kv, dim), values, seen
    (rows of the sequence, len)).  out, lse, sum w|v|, and the largest sum |q k|
    |scale| of a seen key."""
    q = np.asarray(q, dtype=np.float64)
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    absv, big = np.zeros(q.shape), np.zeros(q.shape[:2])
    for row0, k, v, seen in seqs:
        group = q.shape[1] // k.shape[1]
        for i in range(seen.shape[0]):
            if not seen[i].any():
                continue
            for h in range(q.shape[1]):
                kk, vv, row = k[seen[i], h // group], v[seen[i], h // group], q[row0 + i, h]
                x = kk @ row * scale
                w = np.exp(x - x.max())
                z = w.sum()
                out[row0 + i, h], absv[row0 + i, h] = w / z @ vv, w / z @ np.abs(vv)
                lse[row0 + i, h] = x.max() + np.log(z)
                big[row0 + i, h] = (np.abs(kk) @ np.abs(row)).max() * abs(scale)
    return out, lse, absv, big
