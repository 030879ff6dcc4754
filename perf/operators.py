"""Cases of the serving-step operators around a decoding round.

A serving engine that runs draft -> schedule -> verify rounds has, for every round, the tokens whose
target logits verification reads (the anchor and the scheduled draft tokens of each request). Four
operators take them through the target's attention and its sampling rule:

  plan      pages and cache slots of the new tokens, from the requests' lengths
  append    the new tokens' keys and values into the paged cache
  attention the new tokens over a prefix that the whole batch shares (a system prompt) and over each
            request's own pages
  sample /  the target's sampling rule (temperature, top-k, top-p, min-p): one token a row from a given
  truncate  uniform, or the logits with everything outside the kept set masked, for verification

Each has a plain form in elementary torch operations (32 bits) and the library's form. Lengths follow
from the case alone; the order of the requests, the page numbers and all values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

LOG2E = 1.4426950408889634
BF16, FP32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, FP32: torch.float32}


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one round of 128 requests: 1..17 new tokens each (anchor and up to 16 draft tokens)
        {"name": "plan_round", "op": "plan", "R": 128, "new": 17, "cached": 4096, "page": 64},
        # a large fleet's worth of requests with small pages
        {"name": "plan_fleet", "op": "plan", "R": 8192, "new": 17, "cached": 2048, "page": 16},
        # the same round's keys and values
        {"name": "append_round", "op": "append", "R": 128, "new": 17, "cached": 512, "page": 64, "Hkv": 8, "D": 128,
         "dtype": BF16},
        # prompts entering the cache: a chunk of up to 1024 tokens of each of 32 requests
        {"name": "append_prompt", "op": "append", "R": 32, "new": 1024, "cached": 512, "page": 16, "Hkv": 8, "D": 128,
         "dtype": BF16},
        # a single user, a single token: latency
        {"name": "attention_one", "op": "attention", "R": 1, "new": 1, "prefix": 1000, "private": 333, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64},
        # plain decoding, one token a request: bound by the private pages' bytes
        {"name": "attention_decode", "op": "attention", "R": 128, "new": 1, "prefix": 4096, "private": 4096, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64},
        # a scheduled verification round: 1..17 tokens a request, the shared prompt read for all of them
        {"name": "attention_verify", "op": "attention", "R": 128, "new": 17, "prefix": 8192, "private": 2048, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64},
        # a long shared document that ends inside a page, seven query heads a key head, small pages
        {"name": "attention_document", "op": "attention", "R": 64, "new": 9, "prefix": 65553, "private": 500, "Hq": 28,
         "Hkv": 4, "D": 64, "page": 16},
        # one row: latency of the first token
        {"name": "sample_one", "op": "sample", "rows": 1, "V": 32000, "dtype": BF16},
        # one token for each of 128 requests, mixed sampling parameters
        {"name": "sample_decode", "op": "sample", "rows": 128, "V": 129280, "dtype": BF16},
        # target rows of a small-vocabulary round (32 requests, 8 draft tokens), float32, odd row length
        {"name": "truncate_small", "op": "truncate", "rows": 288, "V": 32003, "dtype": FP32},
        # every target row of a round at 128 requests and 16 draft tokens
        {"name": "truncate_verify", "op": "truncate", "rows": 2176, "V": 129280, "dtype": BF16},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "sample", "sample", "truncate"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        return {"op": op, "R": _log(rng, 1, 8192), "new": _log(rng, 1, 17), "cached": _log(rng, 1, 4096), "page": page}
    if op == "append":
        case = {"op": op, "R": _log(rng, 1, 128), "new": _log(rng, 1, 1024), "cached": _log(rng, 1, 512), "page": page,
                "Hkv": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128]), "dtype": rng.choice([BF16, FP32])}
        while case["R"] * case["new"] * case["Hkv"] * case["D"] * (2 if case["dtype"] == BF16 else 4) > 32 * 1024 * 8 * 128 * 2:
            case["new"] = max(1, case["new"] // 2)
            case["R"] = max(1, case["R"] - case["R"] // 4)
        return case
    if op == "attention":
        hkv = rng.choice([1, 2, 4, 8])
        case = {"op": op, "R": _log(rng, 1, 128), "new": _log(rng, 1, 17),
                "prefix": rng.choice([0, 1, 1, 1]) * _log(rng, 16, 65536), "private": _log(rng, 17, 4096),
                "Hq": hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), "Hkv": hkv, "D": rng.choice([64, 128]), "page": page}
        top = {c["name"]: work(c) for c in listed() if c["op"] == op}
        most = {k: max(w[k] for w in top.values()) for k in ("bytes", "flops")}
        while any(work(case)[k] > 0.9 * most[k] for k in most):
            key = "prefix" if case["prefix"] > 4 * case["private"] else "private" if case["private"] > 500 else "R"
            case[key] = max(1, case[key] * 3 // 4)
        return case
    V = _log(rng, 1000, 129280)
    dtype = rng.choice([BF16, FP32])
    rows = _log(rng, 1, 2176 if op == "truncate" else 256)
    while dtype == FP32 and rows * V * 4 > 2176 * 129280 * 2:
        rows = max(1, rows // 2)
    return {"op": op, "rows": rows, "V": V, "dtype": dtype}


def _lengths(case):
    """(new tokens, private tokens before them) of each request: spread evenly over 1..new and 0..cached."""
    R, new = case["R"], case["new"]
    most = case["private"] - case["new"] if case["op"] == "attention" else case["cached"]
    g = np.random.default_rng([R, new, most])
    n = (np.arange(R) * new) // R + 1 if R > 1 else np.array([new])
    c = ((np.arange(R) + 1) * most) // R if R > 1 else np.array([most])
    return g.permutation(n).astype(np.int32), c.astype(np.int32)


def work(case):
    op = case["op"]
    if op in ("sample", "truncate"):
        e = 2 if case["dtype"] == BF16 else 4
        n = case["rows"] * case["V"]
        out = n * e if op == "truncate" else case["rows"] * 8
        return {"bytes": n * e + out + case["rows"] * 24, "flops": 4 * n}
    n, c = (x.astype(np.int64) for x in _lengths(case))
    T = int(n.sum())
    page = case["page"]
    if op == "plan":
        fresh = int(((c + n + page - 1) // page - (c + page - 1) // page).sum())
        return {"bytes": 8 * len(n) + 8 * fresh + 12 * T + 8 * len(n) + 8, "flops": 2 * T}
    if op == "append":
        e = 2 if case["dtype"] == BF16 else 4
        return {"bytes": 4 * T * case["Hkv"] * case["D"] * e + 8 * T, "flops": 0}
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["prefix"]
    seen = int((n * c + n * (n + 1) // 2).sum()) + T * P
    rows = int((n + c).sum()) + P
    return {"bytes": 4 * T * Hq * D + 4 * T * Hq + 4 * rows * Hkv * D, "flops": 4 * seen * Hq * D}


# ---------------------------------------------------------------------------------------------
# inputs

class State:
    pass


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the device workspace that a program keeps next to its streams
        d = _dspark()
        s.ws = (d.new_attention_workspace(s.R, s.T, case["Hq"], case["Hkv"], case["D"]) if s.op == "attention"
                else d.new_workspace(1, 1, 1, 1, d.FP32, 1))
    return s


def _inputs(case, seed):
    s = State()
    s.op, s.case = case["op"], case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(1_000_003 * (seed + 1))
    h = np.random.default_rng([seed, 77])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    if s.op in ("sample", "truncate"):
        N, V, dtype = case["rows"], case["V"], TYPES[case["dtype"]]
        # Zipf-shaped logits with noise, a rank order for each row
        s.logits = torch.empty((N, V), dtype=dtype, device=dev)
        zipf = -1.1 * torch.log1p(torch.arange(V, device=dev, dtype=torch.float32))
        order = torch.randperm(V, generator=g, device=dev)
        turn = torch.from_numpy(h.integers(0, V, N)).to(dev)
        at = torch.arange(V, device=dev)
        for lo in range(0, N, 256):
            rank = order[(at[None, :] + turn[lo:lo + 256, None]) % V]
            s.logits[lo:lo + 256] = (zipf[rank] + 1.5 * torch.randn(rank.shape, generator=g, device=dev)).to(dtype)
        f32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(dev)  # noqa: E731
        s.temperature = f32(h.choice([0.0, 0.6, 0.8, 1.0, 1.0, 1.2], N))
        s.top_k = i32(h.choice([0, 0, 20, 50, 1000], N))
        s.top_p = f32(h.choice([1.0, 0.8, 0.9, 0.95, 0.95], N))
        s.min_p = f32(h.choice([0.0, 0.0, 0.02, 0.05], N))
        s.u = torch.from_numpy(h.random(N)).to(dev)
        s.tokens = torch.empty(N, dtype=torch.int32, device=dev)
        s.prob = torch.empty(N, dtype=torch.float32, device=dev)
        s.out = torch.empty_like(s.logits) if s.op == "truncate" else None
        return s
    page = case["page"]
    n, c = _lengths(case)
    p = h.permutation(len(n))
    n, c = n[p], c[p]
    R, T = len(n), int(n.sum())
    have, need = -(-c // page), -(-(c + n) // page)
    P = case.get("prefix", 0)
    npre = -(-P // page)
    n_pages = int(need.sum()) + npre + 7
    ids = h.permutation(n_pages).astype(np.int32)
    s.page, s.R, s.T, s.prefix = page, R, T, P
    width = int(need.max())
    full = np.zeros((R, width), dtype=np.int32)
    held = np.arange(width)[None, :] < (have if s.op == "plan" else need)[:, None]
    full[held] = ids[npre:npre + int(held.sum())]
    s.table = i32(full)
    s.q_start = i32(np.concatenate([[0], np.cumsum(n)]))
    s.kv_len = i32(c + n)
    s.max_new, s.max_len = int(n.max()), int((c + n).max())
    if s.op == "plan":
        s.free = i32(ids[npre + int(held.sum()):])
        s.cached, s.new = i32(c), i32(n)
        s.position = torch.empty(T, dtype=torch.int32, device=dev)
        s.slots = torch.empty(T, dtype=torch.int64, device=dev)
        s.used = torch.empty(1, dtype=torch.int32, device=dev)
        return s
    Hkv, D = case["Hkv"], case["D"]
    dtype = TYPES[case.get("dtype", BF16)]
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)  # noqa: E731
    s.k_cache, s.v_cache = rand(n_pages, page, Hkv, D), rand(n_pages, page, Hkv, D)
    if s.op == "append":
        s.k, s.v = rand(T, Hkv, D), rand(T, Hkv, D)
        pos = np.concatenate([np.arange(a, a + b) for a, b in zip(c, n)])
        req = np.repeat(np.arange(R), n)
        s.slots = torch.from_numpy(full[req, pos // page].astype(np.int64) * page + pos % page).to(dev)
        return s
    s.q = 1.5 * rand(T, case["Hq"], D)
    s.prefix_pages = i32(ids[:npre])
    s.scale = 1.0 / math.sqrt(D)
    s.out = torch.empty_like(s.q)
    s.lse = torch.empty((T, case["Hq"]), dtype=torch.float32, device=dev)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def _dspark():
    from speculative_decoding_draft_seq_gb300 import dspark
    return dspark


def run(s):
    if not own:
        return {"plan": plain_plan, "append": plain_append, "attention": plain_attention, "sample": plain_sample,
                "truncate": plain_truncate}[s.op](s)
    d = _dspark()
    if s.op == "plan":
        d.page_plan(s.cached, s.new, s.free, s.page, s.table, s.q_start, s.kv_len, s.position, s.slots, s.used, s.ws)
        return s.table, s.q_start, s.kv_len, s.position, s.slots, s.used
    if s.op == "append":
        d.kv_append(s.k, s.v, s.slots, s.k_cache, s.v_cache, s.ws)
        return s.k_cache, s.v_cache
    if s.op == "attention":
        d.prefix_attention(s.q, s.k_cache, s.v_cache, s.prefix_pages, s.prefix, s.table, s.q_start, s.kv_len, s.scale,
                           s.out, s.ws, lse=s.lse)
        return s.out, s.lse
    if s.op == "sample":
        d.sample(s.logits, s.temperature, s.top_k, s.top_p, s.min_p, s.u, s.tokens, s.ws, prob=s.prob)
        return s.tokens, s.prob
    d.truncate(s.logits, s.temperature, s.top_k, s.top_p, s.min_p, s.out, s.ws)
    return s.out


# ---------------------------------------------------------------------------------------------
# plain forms

def plain_plan(s):
    page, cached, new = s.page, s.cached.long(), s.new.long()
    have, need = (cached + page - 1) // page, (cached + new + page - 1) // page
    fresh = need - have
    first = torch.cumsum(fresh, 0) - fresh  # the request's first entry of the list of free pages
    col = torch.arange(s.table.shape[1], device=cached.device)
    is_new = (col >= have[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, max(0, s.free.numel() - 1))
    table = torch.where(is_new, s.free[at], s.table)
    end = torch.cumsum(new, 0)
    tok = torch.arange(s.T, device=cached.device)
    req = torch.searchsorted(end, tok, right=True)
    pos = cached[req] + tok - (end - new)[req]
    slots = table[req, pos // page].long() * page + pos % page
    q_start = torch.cat([end.new_zeros(1), end])
    return table, q_start.int(), (cached + new).int(), pos.int(), slots, fresh.sum().reshape(1).int()


def plain_append(s):
    s.k_cache.view(-1, *s.k.shape[1:])[s.slots] = s.k
    s.v_cache.view(-1, *s.v.shape[1:])[s.slots] = s.v
    return s.k_cache, s.v_cache


def plain_attention(s):
    T, Hq, D = s.q.shape
    Hkv = s.k_cache.shape[2]
    G, R, n = Hq // Hkv, s.R, s.max_new
    q = s.q.float().view(T, Hkv, G, D)
    start, new = s.q_start[:-1].long(), (s.q_start[1:] - s.q_start[:-1]).long()
    # the private part, requests padded to the longest
    i = torch.arange(n, device=q.device)
    tok = (start[:, None] + i).clamp(max=T - 1)
    qp = q[tok].permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D)
    cols = -(-s.max_len // s.page)
    pages = s.table[:, :cols].long()
    k = s.k_cache[pages].view(R, cols * s.page, Hkv, D).permute(0, 2, 3, 1).float()
    v = s.v_cache[pages].view(R, cols * s.page, Hkv, D).permute(0, 2, 1, 3).float()
    x = torch.matmul(qp, k).view(R, Hkv, n, G, -1) * s.scale
    last = s.kv_len[:, None].long() - new[:, None] + i  # the last position that token i sees
    hide = torch.arange(cols * s.page, device=q.device) > last[:, :, None]
    x = x.masked_fill(hide[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    o = torch.matmul(e.view(R, Hkv, n * G, -1), v).view(R, Hkv, n, G, D)
    req = torch.repeat_interleave(torch.arange(R, device=q.device), new, output_size=T)
    own_i = torch.arange(T, device=q.device) - start[req]
    m, z, o = m[req, :, own_i, :, 0], e.sum(-1)[req, :, own_i], o[req, :, own_i]  # [T, Hkv, G(, D)]
    if s.prefix:
        kp = s.k_cache[s.prefix_pages.long()].view(-1, Hkv, D)[:s.prefix].permute(1, 2, 0).float()
        vp = s.v_cache[s.prefix_pages.long()].view(-1, Hkv, D)[:s.prefix].permute(1, 0, 2).float()
        y = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, T * G, D), kp) * s.scale
        mp = y.amax(-1, keepdim=True)
        y = torch.exp(y - mp)
        back = lambda a: a.view(Hkv, T, G, -1).permute(1, 0, 2, 3)  # noqa: E731
        op, zp, mp = back(torch.matmul(y, vp)), back(y.sum(-1, keepdim=True))[..., 0], back(mp)[..., 0]
        top = torch.maximum(m, mp)
        a, b = torch.exp(m - top), torch.exp(mp - top)
        m, z, o = top, z * a + zp * b, o * a[..., None] + op * b[..., None]
    return (o / z[..., None]).reshape(T, Hq, D).to(s.q.dtype), (m + torch.log(z)).reshape(T, Hq)


def _scaled(x, Z):
    """floor(x * Z) for x in [0, 1) on 53 bits and integers Z below 2^60, exactly."""
    k = (x.double() * 2.0 ** 53).floor().long()
    k1, k0 = k >> 27, k & (2 ** 27 - 1)
    z1, z0 = Z >> 29, Z & (2 ** 29 - 1)
    return k1 * z1 * 8 + ((k1 * z0 + 4 * (k0 * z1) + ((k0 * z0) >> 27)) >> 26)


def _kept(s):
    """Weights as 2^-40 integers, the kept set, and the row's first maximum, in vocabulary order."""
    x = s.logits.float() + 0.0
    V = x.shape[1]
    top = x.amax(-1, keepdim=True)
    rate = (LOG2E / s.temperature).clamp(max=1e30)[:, None]
    w = torch.exp2((x - top) * rate)
    w = torch.where(torch.isinf(x), torch.zeros_like(w), w)
    fx = (w * 2.0 ** 40).long()
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices  # ties: the lowest index first
    sw, sf = w.gather(-1, order), fx.gather(-1, order)
    rank = torch.arange(V, device=x.device)
    k = torch.where(s.top_k > 0, s.top_k, V)[:, None]
    keep = rank < k
    sf1 = torch.where(keep, sf, torch.zeros_like(sf))
    before = torch.cumsum(sf1, -1) - sf1
    limit = _scaled(s.top_p.clamp(0, 1 - 2.0 ** -24), sf1.sum(-1)).clamp(min=1)[:, None]
    keep &= (before < limit) | (s.top_p >= 1)[:, None]
    keep &= sw >= s.min_p.clamp(0, 1)[:, None]
    keep &= x.gather(-1, order) > -math.inf
    greedy = (s.temperature <= 0)[:, None]
    keep = torch.where(greedy, rank == 0, keep)
    kept = torch.zeros_like(keep).scatter_(-1, order, keep)
    return fx, kept, order[:, 0]


def plain_sample(s):
    fx, kept, first = _kept(s)
    fx = torch.where(kept, fx, torch.zeros_like(fx))
    cum = torch.cumsum(fx, -1)
    Z = cum[:, -1]
    token = (cum > _scaled(s.u, Z)[:, None]).int().argmax(-1)
    prob = (fx.gather(-1, token[:, None])[:, 0].double() / Z.double()).float()
    greedy = s.temperature <= 0
    return torch.where(greedy, first, token).int(), torch.where(greedy, torch.ones_like(prob), prob)


def plain_truncate(s):
    _, kept, _ = _kept(s)
    return torch.where(kept, s.logits, torch.full_like(s.logits, torch.finfo(s.logits.dtype).min))


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(_inputs(case, seed))
    if case["op"] == "sample":
        return _exact_sample(_inputs(case, seed))
    return None  # page numbers, copies and selections: nothing is rounded


def _exact_attention(s):
    T, Hq, D = s.q.shape
    Hkv = s.k_cache.shape[2]
    outs, lses = [], []
    start, length = s.q_start.tolist(), s.kv_len.tolist()
    pre = s.prefix_pages.long()
    kp = s.k_cache[pre].reshape(-1, Hkv, D)[:s.prefix].double()
    vp = s.v_cache[pre].reshape(-1, Hkv, D)[:s.prefix].double()
    for r in range(s.R):
        n, L = start[r + 1] - start[r], length[r]
        pages = s.table[r, :-(-L // s.page)].long()
        k = torch.cat([kp, s.k_cache[pages].reshape(-1, Hkv, D)[:L].double()])
        v = torch.cat([vp, s.v_cache[pages].reshape(-1, Hkv, D)[:L].double()])
        q = s.q[start[r]:start[r + 1]].double().view(n, Hkv, Hq // Hkv, D)
        x = torch.einsum("ihgd,jhd->hgij", q, k) * s.scale
        i, j = torch.arange(n, device=x.device)[:, None], torch.arange(s.prefix + L, device=x.device)[None, :]
        x = torch.where(j - s.prefix <= L - n + i, x, torch.full_like(x, -math.inf))
        lse = torch.logsumexp(x, -1)
        o = torch.einsum("hgij,jhd->ihgd", torch.exp(x - lse[..., None]), v)
        outs.append(o.reshape(n, Hq, D))
        lses.append(lse.permute(2, 0, 1).reshape(n, Hq))
    return torch.cat(outs), torch.cat(lses)


def _exact_sample(s):
    probs = []
    V = s.logits.shape[1]
    for r in range(s.logits.shape[0]):
        x = s.logits[r].double()
        T = float(s.temperature[r])
        if T <= 0:
            probs.append(torch.ones((), dtype=torch.float64, device=x.device))
            continue
        y, order = torch.sort(x, descending=True, stable=True)
        p = torch.softmax(y / T, 0)
        k = int(s.top_k[r])
        p[k if k > 0 else V:] = 0
        total = p.sum()
        keep = (p > 0) & (torch.cumsum(p, 0) - p < float(s.top_p[r]) * total if float(s.top_p[r]) < 1 else p > 0)
        keep &= p >= float(s.min_p[r]) * p[0]
        q = torch.zeros_like(p)
        q[order[keep]] = p[keep]
        q /= q.sum()
        at = int(torch.searchsorted(torch.cumsum(q, 0), s.u[r].double().reshape(1), right=True)[0])
        probs.append(q[min(at, V - 1)])
    return None, torch.stack(probs).double()
