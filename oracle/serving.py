"""Oracle of the target's side of a round in a serving engine: cache pages and slots, attention over a
shared prefix and private pages, and the sampling rule. Plain numpy in float64 (integers where the
definition has integers), one request, row or token at a time."""
import itertools
import math

import numpy as np


def page_plan(cached, new, free, page, table, capacity):
    """Block table, starts, lengths, positions, slots and pages used; short lists leave -1. Of the new tokens those that
    fit the capacity are planned, in request order. The list of free pages ends at its first negative id."""
    free = [int(x) for x in itertools.takewhile(lambda x: x >= 0, free)]
    table = np.array(table, dtype=np.int64)
    R, width = table.shape
    taken, tok, short = 0, 0, sum(max(0, int(n)) for n in new) > capacity
    q_start, kv_len, positions, slots = [], [], [], []
    for r in range(R):
        q_start.append(tok)
        c, n = int(cached[r]), min(int(new[r]), capacity - tok)
        for col in range(-(-c // page), -(-(c + n) // page)):
            page_id = free[taken] if taken < len(free) else -1
            short |= page_id < 0 or col >= width
            taken += 1
            if col < width:
                table[r, col] = page_id
        for pos in range(c, c + n):
            col = pos // page
            page_id = int(table[r, col]) if col < width else -1
            positions.append(pos)
            slots.append(-1 if page_id < 0 else page_id * page + pos % page)
            tok += 1
        kv_len.append(c + n)
    q_start.append(tok)
    pad = [-1] * (capacity - tok)
    return {"table": table, "q_start": q_start, "kv_len": kv_len, "positions": positions + pad, "slots": slots + pad, "used": min(taken, len(free)), "short": short}


def attention(q, k_cache, v_cache, prefix_pages, prefix_len, table, q_start, kv_len, scale):
    """(out, lse, spread, score_error) in float64. spread: sum_j weight_j |v_j| (what a relative error of the weights
    multiplies); score_error [T, Hq]: a bound on the error of a float32 score, accumulated in any order."""
    T, Hq, D = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hkv
    q = q.astype(np.float64)
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, err = np.full((T, Hq), -np.inf), np.zeros((T, Hq))

    def rows(cache, pages, length, h):
        return cache[pages[:-(-length // page)], :, h].reshape(-1, D)[:length].astype(np.float64)

    for r in range(len(kv_len)):
        n, L = q_start[r + 1] - q_start[r], int(kv_len[r])
        for h in range(Hkv if n else 0):
            k = np.concatenate([rows(k_cache, prefix_pages, prefix_len, h), rows(k_cache, table[r], L, h)])
            v = np.concatenate([rows(v_cache, prefix_pages, prefix_len, h), rows(v_cache, table[r], L, h)])
            for i in range(n):
                t, seen = q_start[r] + i, prefix_len + max(0, L - n + i + 1)
                if seen == 0:
                    continue
                for g in range(h * G, (h + 1) * G):
                    x = k[:seen] @ q[t, g] * scale
                    m = x.max()
                    e = np.exp(x - m)
                    w = e / e.sum()
                    out[t, g], spread[t, g] = w @ v[:seen], w @ np.abs(v[:seen])
                    lse[t, g] = m + math.log(e.sum())
                    err[t, g] = ((np.abs(k[:seen]) @ np.abs(q[t, g])).max() * scale * (D + 2) + np.abs(x).max() * 4) * 2.0 ** -24
    return out, lse, spread, err


def rule(x, temperature, top_k, top_p, min_p):
    """(kept mask, weights relative to the maximum, margin) of one row. margin: how far, relative to the
    quantities compared, the nearest comparison is from changing."""
    x = np.asarray(x, dtype=np.float64)
    V = len(x)
    order = np.lexsort((np.arange(V), -x))
    kept = np.zeros(V, dtype=bool)
    if not temperature > 0:
        kept[order[0]] = True
        return kept, kept.astype(np.float64), np.inf
    with np.errstate(invalid="ignore"):
        w = np.where(np.isneginf(x), 0.0, np.exp2((x - x[order[0]]) * min(math.log2(math.e) / temperature, 1e30)))
    s = w[order]
    keep = np.ones(V, dtype=bool)
    if 0 < top_k < V:
        keep[top_k:] = False
    margin = np.inf
    if top_p < 1:
        before = np.cumsum(np.where(keep, s, 0.0)) - s
        S = s[keep].sum()
        inside = before < max(top_p * S, 2.0 ** -40)
        if keep[1:].any():
            margin = np.abs(before[1:][keep[1:]] - top_p * S).min() / S
        keep &= inside
    if min_p > 0:
        margin = min(margin, np.abs(s - min(min_p, 1.0))[1:].min(initial=np.inf) / min_p)
        keep &= s >= min(min_p, 1.0)
    kept[order[keep]] = True
    kept &= x > -np.inf
    return kept, w, margin


def draw(kept, w, u):
    """(token, probability, margin) of the inverse-CDF draw in vocabulary order."""
    c = np.cumsum(np.where(kept, w, 0.0))
    Z = c[-1]
    v = int(np.searchsorted(c, u * Z, side="right"))
    return v, w[v] / Z, np.abs(c - u * Z).min() / Z


def exact_masses(x, rate):
    """floor(2^((x - max) rate) 2^40) as Python integers where (x - max) rate is a whole number."""
    top = max(x)
    return [0 if a == -math.inf or (top - a) * rate > 40 else 1 << int(40 - (top - a) * rate) for a in x]


def exact_rule(x, rate, top_k, top_p, min_p, u=None):
    """The rule in exact integers for rows whose weights are powers of two: (kept list, token, probability)."""
    V, fx = len(x), exact_masses(x, rate)
    order = sorted(range(V), key=lambda v: (-x[v], v))
    if 0 < top_k < V:
        order = order[:top_k]
    if top_p < 1:
        limit, before, cut = max(1, int(top_p * 2 ** 53) * sum(fx[v] for v in order) >> 53), 0, []
        for v in order:
            if before < limit:
                cut.append(v)
            before += fx[v]
        order = cut
    top = max(x)
    kept = sorted(v for v in order if 2.0 ** -min((top - x[v]) * rate, 1000.0) >= min(max(min_p, 0.0), 1.0) and x[v] > -math.inf)
    if u is None:
        return kept, None, None
    Z = sum(fx[v] for v in kept)
    t, c = int(u * 2 ** 53) * Z >> 53, 0
    for v in kept:
        c += fx[v]
        if c > t:
            return kept, v, fx[v] / Z
