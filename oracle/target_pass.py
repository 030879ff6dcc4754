"""Oracle of what follows the target's pass over a round's tokens: probabilities of rows of logits,
verification of drafted tokens from given uniforms, pages of the cache, and distillation from a teacher's
top logits. Plain numpy in float64 and Python integers, one row, request or page at a time.

Pinned in tests/test_oracle_target_pass.py: the output law of a verified block by enumeration of its
uniforms, the gradients by differences, the page lists by what each row reads through its table."""
import itertools
import math
from fractions import Fraction

import numpy as np


def softmax(x, temperature):
    """(probabilities, exponents in octaves) of one row; a row without a finite maximum gives zeros."""
    x = np.asarray(x, dtype=np.float64)
    M = x.max()
    if not np.isfinite(M):
        return np.zeros_like(x), np.zeros_like(x)
    if not temperature > 0:
        return (np.arange(len(x)) == np.argmax(x)).astype(np.float64), np.zeros_like(x)
    rate = min(math.log2(math.e) / temperature, 1e30) if temperature < math.inf else 0.0
    with np.errstate(invalid="ignore"):
        y = np.where(np.isneginf(x), -np.inf, (x - M) * rate)
    w = np.exp2(y)
    return w / w.sum(), np.where(np.isneginf(y), 0.0, y)


# ---------------------------------------------------------------------------------------------
# verification

def masses(w):
    """floor(min(w, 1) 2^40) of float32 values as Python integers; NaN and negative ones 0."""
    return [0 if not x > 0 else int(Fraction(min(float(x), 1.0)) * 2 ** 40) for x in w]


def draw(w, u):
    """The first index whose mass up to and including it exceeds floor(u Z); -1 without mass."""
    m = masses(w)
    Z = sum(m)
    if Z == 0:
        return -1
    goal = int(Fraction(min(max(float(u), 0.0), 1.0 - 2.0 ** -53)) * 2 ** 53) * Z >> 53
    c = 0
    for v, x in enumerate(m):
        c += x
        if c > goal:
            return v
    raise AssertionError


def verify_probs(target, q_start, draft, tokens, u):
    """(out_tokens, accepted_len, p_tok); target [T, V] and draft [R, gamma, V] (or None) float32 values."""
    R, gamma = tokens.shape
    V = target.shape[1]
    out, acc, p_tok = np.full((R, gamma + 1), -1), np.zeros(R, dtype=int), np.zeros((R, gamma), dtype=np.float32)
    for r in range(R):
        first, last = int(q_start[r]), int(q_start[r + 1])
        if first < 0 or last <= first or last > len(target):
            continue
        L = min(last - first - 1, gamma)
        ok = []
        for k in range(L):
            x = int(tokens[r, k])
            if not 0 <= x < V:
                ok.append(False)
                continue
            p_tok[r, k] = target[first + k, x]
            q = np.float32(1.0) if draft is None else draft[r, k, x]
            ok.append(bool(np.float64(u[r, k]) * np.float64(q) < np.float64(p_tok[r, k])))
        a = ok.index(False) if False in ok else L
        row = target[first + a].astype(np.float32)
        w = row
        if a < L and 0 <= tokens[r, a] < V:
            q = draft[r, a].astype(np.float32) if draft is not None else (np.arange(V) == tokens[r, a]).astype(np.float32)
            with np.errstate(invalid="ignore"):
                w = row - q
        new = draw(w, u[r, gamma])
        if new < 0:
            new = draw(row, u[r, gamma])
        out[r, :a] = tokens[r, :a]
        out[r, a] = new
        acc[r] = a
    return out, acc, p_tok


# ---------------------------------------------------------------------------------------------
# pages

def _row(table, kv_len, r, page):
    width = len(table[r])
    n = min(max(int(kv_len[r]), 0), width * page)
    return [int(x) for x in table[r][:-(-n // page)]]


def page_collect(table, kv_len, page, n_pages, pinned=()):
    """(refs, free list padded with -1, number of free pages)."""
    refs = [0] * n_pages
    for x in [x for r in range(len(table)) for x in _row(table, kv_len, r, page)] + list(pinned):
        if 0 <= x < n_pages:
            refs[x] += 1
    free = [x for x in range(n_pages) if refs[x] == 0]
    return refs, free + [-1] * (n_pages - len(free)), len(free)


def page_fork(table, kv_len, parent, fork_len, page, n_pages, free, pinned=()):
    """Dictionary of new_table, new_len, src, dst, tokens, used. The list of free pages ends at its first negative id."""
    width, rows, lens = len(table[0]), [], []
    free = [int(x) for x in itertools.takewhile(lambda x: x >= 0, free)]
    for i, q in enumerate(parent):
        have = 0 if not 0 <= q < len(table) else min(max(int(kv_len[q]), 0), width * page)
        n = have if fork_len is None else min(max(int(fork_len[i]), 0), have)
        lens.append(n)
        rows.append([int(x) for x in table[q][:-(-n // page)]] if n else [])
    inside = lambda x: 0 <= x < n_pages  # noqa: E731
    full = set(pinned) | {x for row, n in zip(rows, lens) for x in row[:n // page]}
    ended, taken, wanted = set(), 0, 0
    src, dst, tokens = [], [], []
    for row, n in zip(rows, lens):
        rest = n % page
        if not rest or not inside(row[-1]) or (row[-1] not in full and row[-1] not in ended):
            if rest:
                ended.add(row[-1])
            src.append(-1), dst.append(-1), tokens.append(0)
            continue
        to = free[wanted] if wanted < len(free) else -1
        wanted += 1
        taken = min(wanted, len(free))
        src.append(row[-1] if to >= 0 else -1), dst.append(to), tokens.append(rest if to >= 0 else 0)
        row[-1] = to
    return {"new_table": [row + [-1] * (width - len(row)) for row in rows], "new_len": lens, "src": src, "dst": dst,
            "tokens": tokens, "used": taken}


def page_compact(table, kv_len, page, n_pages, pinned=()):
    """Dictionary of new_table, new_pinned, src, dst, n_live."""
    refs, _, _ = page_collect(table, kv_len, page, n_pages, pinned)
    live = [x for x in range(n_pages) if refs[x]]
    m = len(live)
    src, dst = [x for x in live if x >= m], [x for x in range(m) if not refs[x]]
    name = dict(zip(src, dst))
    width, pad = len(table[0]), [-1] * (n_pages // 2 - len(src))
    rows = [[name.get(x, x) for x in _row(table, kv_len, r, page)] for r in range(len(table))]
    return {"new_table": [row + [-1] * (width - len(row)) for row in rows], "new_pinned": [name.get(x, x) for x in pinned],
            "src": src + pad, "dst": dst + pad, "n_live": m}


# ---------------------------------------------------------------------------------------------
# distillation

def distill(x, ids, teacher, tau, lse=None):
    """(loss, d loss / d x, parts) of one row; parts: s, p over the vocabulary, p_rest, s_rest, octaves below the maximum.
    The rest's logarithm and its entries' shares in it are formed from its own maximum: s_rest may be far below float64's range."""
    x, t = np.asarray(x, dtype=np.float64), np.asarray(teacher, dtype=np.float64) / tau
    V = len(x)
    keep = [j for j, v in enumerate(ids) if 0 <= v < V]
    M = x.max()
    with np.errstate(divide="ignore"):
        ln_s = x / tau - (M / tau + math.log(np.exp((x - M) / tau).sum()))
    s = np.exp(ln_s)
    p, p_rest, s_rest, loss = np.zeros(V), 0.0, 0.0, 0.0
    named = np.zeros(V, dtype=bool)
    named[[int(ids[j]) for j in keep]] = True
    listed = [t[j] for j in keep]
    if lse is not None:
        shift, p_rest = float(lse), 1.0
    else:
        top = max(listed, default=-math.inf)
        if top > -math.inf:
            t = t - top  # (of masked entries a sum's logarithm would vanish beside the largest)
        shift = math.log(sum(math.exp(a - top) for a in listed)) if top > -math.inf else None
    for j in keep if shift is not None else []:
        q = math.exp(t[j] - shift)
        if q > 0:
            loss += q * (t[j] - shift - ln_s[ids[j]])
        p[ids[j]] += q
    if lse is not None:
        p_rest, s_rest = max(0.0, 1.0 - p.sum()), s[~named].sum()
        x_out = np.where(named, -np.inf, x)
        top = x_out.max()
        if p_rest > 0 and top > -math.inf:
            out = np.exp((x_out - top) / tau)
            loss += p_rest * (math.log(p_rest) - ln_s[np.argmax(x_out)] - math.log(out.sum()))
        else:
            p_rest = 0.0
    grad = s * (p.sum() + p_rest) - p
    if p_rest > 0:
        grad = grad - p_rest * (out / out.sum())
    return loss, grad / tau, {"s": s, "p": p, "p_rest": p_rest, "s_rest": s_rest, "named": named,
                              "below": np.where(np.isneginf(x), 0.0, (M - x) / tau)}
