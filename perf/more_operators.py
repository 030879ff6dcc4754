"""Cases of the operators that follow the target's pass over a round's tokens.

Once the target has run, its rows of logits become probabilities, these decide which drafted tokens
stand, the cache follows that decision, and the rows' largest entries teach the drafter:

  probs    softmax of rows of logits, one temperature a row
  verify   drafted tokens against the target's probabilities, from given uniforms: any drafter, with
           its own rows of probabilities or without (a table lookup)
  collect  how many requests hold each page of the cache, and the list of the free ones
  fork     block-table rows that continue other rows, pages shared, and copies of the pages they write next
  compact  the live pages moved to the front of the cache
  distill  the divergence of a drafter's rows from a teacher's top logits, and its gradient

Each has a plain form in elementary torch operations and the library's form. Lengths and which row
forks which follow from the case alone; page numbers, the order of rows and all values follow from the seed.
"""
import functools
import math

import numpy as np
import torch

own = False

LOG2E = 1.4426950408889634
BF16, FP32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
SIZES = {BF16: 2, FP32: 4}


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the first token of one request
        {"name": "probs_one", "op": "probs", "rows": 1, "V": 32000, "dtype": BF16, "out": FP32},
        # the target rows of a scheduled round: 128 requests, 1..17 rows each
        {"name": "probs_round", "op": "probs", "rows": 1152, "V": 129280, "dtype": BF16, "out": FP32},
        # one user, four tokens looked up in the prompt: no rows of the drafter's own
        {"name": "verify_lookup", "op": "verify", "R": 1, "gamma": 4, "V": 32000, "dtype": FP32, "draft": False},
        # a scheduled round of 128 requests, up to 16 tokens of a small model each
        {"name": "verify_round", "op": "verify", "R": 128, "gamma": 16, "V": 129280, "dtype": FP32, "draft": True},
        # the holders of a round's pages, after the rejected tokens are gone; four samples of each prompt
        {"name": "collect_round", "op": "collect", "R": 128, "cached": 4096, "page": 64, "group": 4},
        # a fleet's worth of requests with small pages
        {"name": "collect_fleet", "op": "collect", "R": 8192, "cached": 2048, "page": 16, "group": 4},
        # a second, third and fourth sample of one short prompt
        {"name": "fork_one", "op": "fork", "from": 1, "rows": 4, "cut": 0, "cached": 333, "page": 16, "group": 1,
         "layers": 2, "Hkv": 2, "D": 64, "dtype": BF16},
        # four samples of each of 32 prompts
        {"name": "fork_samples", "op": "fork", "from": 32, "rows": 128, "cut": 0, "cached": 4000, "page": 64, "group": 1,
         "layers": 2, "Hkv": 8, "D": 128, "dtype": BF16},
        # eight short requests in a small cache
        {"name": "compact_few", "op": "compact", "R": 8, "cached": 300, "page": 16, "group": 1, "layers": 2, "Hkv": 2,
         "D": 64, "dtype": BF16},
        # a cache a third empty, brought to the front of its pool
        {"name": "compact_round", "op": "compact", "R": 128, "cached": 1024, "page": 16, "group": 4, "layers": 2,
         "Hkv": 8, "D": 128, "dtype": BF16},
        # a few rows with the teacher's normaliser, float32, odd row length
        {"name": "distill_few", "op": "distill", "rows": 32, "V": 32003, "K": 20, "dtype": FP32, "rest": True,
         "back": True},
        # every drafted position of a round at 128 requests and 16 tokens, the teacher's top 64
        {"name": "distill_round", "op": "distill", "rows": 2048, "V": 129280, "K": 64, "dtype": BF16, "rest": False,
         "back": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["probs", "verify", "verify", "collect", "fork", "compact", "distill", "distill"])
    page = rng.choice([16, 32, 64, 128])
    cache = {"layers": rng.choice([1, 2, 3]), "Hkv": rng.choice([1, 2, 4, 8]), "D": rng.choice([64, 128]),
             "dtype": rng.choice([BF16, FP32])}
    if op == "probs":
        case = {"op": op, "rows": _log(rng, 1, 1152), "V": _log(rng, 1000, 129280), "dtype": rng.choice([BF16, FP32]),
                "out": rng.choice([BF16, FP32])}
        key = "rows"
    elif op == "verify":
        case = {"op": op, "R": _log(rng, 1, 128), "gamma": _log(rng, 1, 16), "V": _log(rng, 1000, 129280),
                "dtype": rng.choice([BF16, FP32]), "draft": rng.choice([True, True, False])}
        key = "R"
    elif op == "collect":
        case = {"op": op, "R": _log(rng, 1, 8192), "cached": _log(rng, 1, 4096), "page": page,
                "group": rng.choice([1, 2, 4])}
        key = "R"
    elif op == "fork":
        few = _log(rng, 1, 32)
        case = {"op": op, "from": few, "rows": _log(rng, few, 128), "cut": rng.choice([0, 0, 17, 500]),
                "cached": _log(rng, 16, 4096), "page": page, "group": rng.choice([1, 2]), **cache}
        key = "cached"
    elif op == "compact":
        case = {"op": op, "R": _log(rng, 1, 128), "cached": _log(rng, 16, 1024), "page": page,
                "group": rng.choice([1, 2, 4]), **cache}
        key = "R"
    else:
        case = {"op": op, "rows": _log(rng, 1, 2048), "V": _log(rng, 1000, 129280), "K": _log(rng, 1, 256),
                "dtype": rng.choice([BF16, FP32]), "rest": rng.choice([True, False]),
                "back": rng.choice([True, True, False])}
        key = "rows"
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    held = max(_held(c) for c in listed() if c["op"] == op)
    while work(case)["bytes"] > 0.95 * most or _held(case) > held:
        case[key] = max(1, case[key] * 3 // 4)
        if op == "fork":
            case["layers"] = 1
    return case


def _held(case):
    """Bytes of the inputs, which may be much more than a pass reads."""
    if case["op"] == "verify":
        return case["R"] * case["V"] * SIZES[case["dtype"]] * (case["gamma"] + 1) * 2
    if case["op"] in ("fork", "compact"):
        return _pages(case) * case["page"] * case["layers"] * case["Hkv"] * case["D"] * 2 * SIZES[case["dtype"]]
    return 0


@functools.lru_cache(maxsize=64)
def _layout_of(R, cached, page, group):
    """(lengths, block table) of R requests, pages numbered from 0 in order: lengths spread evenly over 0..cached;
    the requests of a group share the first half of the shortest one's full pages."""
    g = np.random.default_rng([R, cached, page, group])
    c = g.permutation(((np.arange(R) + 1) * cached) // R)
    need = -(-c // page)
    lead = np.arange(R) // group * group
    short = np.minimum.reduceat(c, np.arange(0, R, group))[np.arange(R) // group]
    shared = np.where(np.arange(R) == lead, 0, short // page // 2)
    mine = need - shared
    start = np.cumsum(mine) - mine
    col = np.arange(max(1, int(need.max())))
    table = np.where(col < shared[:, None], start[lead][:, None] + col, start[:, None] + col - shared[:, None])
    return c, np.where(col < need[:, None], table, -1)


def _layout(case):
    return _layout_of(case["from"] if case["op"] == "fork" else case["R"], case["cached"], case["page"], case["group"])


def _pages(case):
    """Pages of the cache: half as many again as are held, and some."""
    live = int(_layout(case)[1].max()) + 1
    return live + live // 2 + 8 + (case["rows"] if case["op"] == "fork" else 0)


def _forks(case):
    """(parent, length) of each new row: samples of every request, or beams that drop, double and cut rows."""
    c, _ = _layout(case)
    n, few = case["rows"], case["from"]
    if not case["cut"]:
        parent = np.arange(n) * few // n
        return parent, c[parent]
    g = np.random.default_rng([n, few, case["cut"]])
    parent = g.integers(-1, few, n)
    return parent, np.where(parent < 0, 0, np.maximum(0, c[parent] - g.integers(0, case["cut"] + 1, n)))


def _lengths(case):
    """Rows of each request of a round (drafts + 1), spread evenly over 1..gamma + 1."""
    R, n = case["R"], case["gamma"] + 1
    if R == 1:
        return np.array([n])
    return np.random.default_rng([R, n]).permutation((np.arange(R) * n) // R + 1)


def work(case):
    op = case["op"]
    if op == "probs":
        n = case["rows"] * case["V"]
        return {"bytes": n * (SIZES[case["dtype"]] + SIZES[case["out"]]) + 4 * case["rows"], "flops": 4 * n}
    if op == "verify":
        # every request reads one row of the target, and one of the drafter where a draft is rejected (at this noise
        # three drafts in four are accepted); a lookup has no rows
        n = _lengths(case)
        rows = case["R"] + (float((1 - 0.75 ** (n - 1)).sum()) if case["draft"] else 0)
        T = int(n.sum())
        return {"bytes": int(rows * case["V"]) * SIZES[case["dtype"]] + T * (4 + 8 + 2 * SIZES[case["dtype"]] + 8),
                "flops": int(3 * rows * case["V"])}
    if op == "distill":
        n = case["rows"] * case["V"]
        return {"bytes": n * SIZES[case["dtype"]] * (2 if case["back"] else 1) + case["rows"] * (8 * case["K"] + 12),
                "flops": (8 if case["back"] else 4) * n}
    c, table = _layout(case)
    entries, n_pages = int((table >= 0).sum()), _pages(case)
    live = int(table.max()) + 1
    if op == "collect":
        return {"bytes": 4 * (entries + len(c) + n_pages + n_pages - live), "flops": entries + n_pages}
    row = 2 * case["layers"] * case["Hkv"] * case["D"] * SIZES[case["dtype"]]  # K and V of a token
    if op == "compact":
        moves = live * (n_pages - live) // n_pages
        return {"bytes": 8 * entries + 8 * moves + 2 * moves * case["page"] * row, "flops": entries + n_pages}
    parent, length = _forks(case)
    need = -(-length // case["page"])
    copied, seen = 0, set()
    full = {int(x) for i in range(len(parent)) if parent[i] >= 0
            for x in table[parent[i], :length[i] // case["page"]]}
    for i in range(len(parent)):
        if length[i] % case["page"]:
            x = int(table[parent[i], length[i] // case["page"]])
            if x in full or x in seen:
                copied += int(length[i] % case["page"])
            seen.add(x)
    return {"bytes": 8 * int(need.sum()) + 20 * len(parent) + 2 * copied * row, "flops": int(need.sum())}


# ---------------------------------------------------------------------------------------------
# inputs

class State:
    pass


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the device workspace that a program keeps next to its streams
        d = _dspark()
        s.ws = d.new_page_workspace(s.n_pages) if s.op in ("collect", "fork", "compact") else \
            d.new_workspace(1, 1, 1, 1, d.FP32, 1)
    return s


def _logit_rows(g, n, V, sd):
    """Zipf-shaped rows with noise, a rank order for each, in float32."""
    dev = "cuda"
    zipf = -1.1 * torch.log1p(torch.arange(V, device=dev, dtype=torch.float32))
    order = torch.randperm(V, generator=g, device=dev)
    turn = torch.randint(V, (n, 1), generator=g, device=dev)
    at = torch.arange(V, device=dev)
    return zipf[order[(at + turn) % V]] + sd * torch.randn((n, V), generator=g, device=dev)


def _softmax(x):
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _inputs(case, seed):
    s = State()
    s.op, s.case = case["op"], case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(2_000_003 * (seed + 1))
    h = np.random.default_rng([seed, 99])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    empty = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
    dtype = TYPES[case.get("dtype", BF16)]
    if s.op == "probs":
        N, V = case["rows"], case["V"]
        s.logits = empty(N, V, dtype=dtype)
        for lo in range(0, N, 256):
            s.logits[lo:lo + 256] = _logit_rows(g, min(256, N - lo), V, 1.5).to(dtype)
        s.temperature = torch.from_numpy(h.choice([0.0, 0.6, 0.8, 1.0, 1.0, 1.2], N).astype(np.float32)).to(dev)
        s.probs = empty(N, V, dtype=TYPES[case["out"]])
        return s
    if s.op == "verify":
        R, G, V = case["R"], case["gamma"], case["V"]
        n = h.permutation(_lengths(case))
        start = np.concatenate([[0], np.cumsum(n)])
        s.T = int(start[-1])
        s.q_start = i32(start)
        s.target = empty(s.T, V, dtype=dtype)
        s.draft = empty(R, G, V, dtype=dtype) if case["draft"] else None
        s.tokens = empty(R, G)
        for r in range(R):
            x = _logit_rows(g, G + 1, V, 1.5)
            s.target[start[r]:start[r + 1]] = _softmax(x[:n[r]]).to(dtype)
            q = _softmax(x[:G] + 0.4 * torch.randn((G, V), generator=g, device=dev))
            if case["draft"]:
                s.draft[r] = q.to(dtype)
                s.tokens[r] = torch.multinomial(q, 1, generator=g)[:, 0].int()
            else:
                s.tokens[r] = q.argmax(-1).int()
        s.u = torch.from_numpy(h.random((R, G + 1))).to(dev)
        s.out_tokens, s.accepted, s.p_tok = empty(R, G + 1), empty(R), empty(R, G, dtype=torch.float32)
        return s
    if s.op == "distill":
        N, V, K = case["rows"], case["V"], min(case["K"], case["V"])
        s.tau = 1.5
        s.logits = empty(N, V, dtype=dtype)
        s.ids, s.teacher = empty(N, K), empty(N, K, dtype=torch.float32)
        s.lse = empty(N, dtype=torch.float32) if case["rest"] else None
        for lo in range(0, N, 256):
            x = _logit_rows(g, min(256, N - lo), V, 1.5)
            at = slice(lo, lo + 256)
            s.teacher[at], ids = torch.topk(x, K)
            s.ids[at] = ids.int()
            if case["rest"]:
                s.lse[at] = torch.logsumexp(x.double() / s.tau, -1).float()
            s.logits[at] = (x + 0.5 * torch.randn(x.shape, generator=g, device=dev)).to(dtype)
        s.ids[1::7, K // 2 + 1:] = -1  # shorter lists are padded
        w = np.full(N, 1.0 / N, dtype=np.float32)
        w[3::16] = 0.0  # positions past a request's end
        s.weight = torch.from_numpy(w).to(dev)
        s.loss = empty(N, dtype=torch.float32)
        s.grad = torch.empty_like(s.logits) if case["back"] else None
        return s
    c, table = _layout(case)
    page, s.n_pages = case["page"], _pages(case)
    ids = h.permutation(s.n_pages)
    s.page, s.R, s.width = page, len(c), table.shape[1]
    s.table = i32(np.where(table >= 0, ids[table], -1))
    s.kv_len = i32(c)
    n_pin = min(3, s.n_pages - int(table.max()) - 1)  # a system prompt's pages
    s.pinned = i32(ids[s.n_pages - n_pin:])
    if s.op == "collect":
        s.refs, s.free, s.n_free = empty(s.n_pages), empty(s.n_pages), empty(1)
        return s
    shape = (case["layers"], s.n_pages, page, case["Hkv"], case["D"])
    s.k, s.v = (torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype) for _ in range(2))
    if s.op == "compact":
        s.new_table, s.new_pinned, s.n_live = empty(s.R, s.width), empty(n_pin), empty(1)
        s.src, s.dst = empty(s.n_pages // 2), empty(s.n_pages // 2)
        return s
    parent, length = _forks(case)
    n = len(parent)
    s.parent, s.length = i32(parent), i32(length)
    s.free = i32(np.sort(ids[int(table.max()) + 1:s.n_pages - n_pin]))
    s.new_table, s.new_len, s.used = empty(n, s.width), empty(n), empty(1)
    s.src, s.dst, s.tokens = empty(n), empty(n), empty(n)
    return s


# ---------------------------------------------------------------------------------------------
# one pass

def _dspark():
    from speculative_decoding_draft_seq_gb300 import dspark
    return dspark


def run(s):
    if not own:
        return {"probs": plain_probs, "verify": plain_verify, "collect": plain_collect, "fork": plain_fork,
                "compact": plain_compact, "distill": plain_distill}[s.op](s)
    d = _dspark()
    if s.op == "probs":
        d.probabilities(s.logits, s.temperature, s.probs, s.ws)
        return s.probs
    if s.op == "verify":
        d.verify_probs(s.target, s.q_start, s.draft, s.tokens, s.u, s.out_tokens, s.accepted, s.p_tok, s.ws)
        return s.out_tokens, s.accepted, s.p_tok
    if s.op == "collect":
        d.page_collect(s.table, s.kv_len, s.page, s.refs, s.free, s.n_free, s.ws, pinned=s.pinned)
        return s.refs, s.free, s.n_free
    if s.op == "fork":
        d.page_fork(s.table, s.kv_len, s.parent, s.length, s.page, s.n_pages, s.free, s.new_table, s.new_len, s.src, s.dst,
                    s.tokens, s.used, s.ws, pinned=s.pinned)
        d.page_copy(s.src, s.dst, s.k, s.v, s.ws, tokens=s.tokens)
        return s.new_table, s.new_len, s.src, s.dst, s.tokens, s.used, s.k, s.v
    if s.op == "compact":
        d.page_compact(s.table, s.kv_len, s.page, s.n_pages, s.new_table, s.src, s.dst, s.n_live, s.ws, pinned=s.pinned,
                       new_pinned=s.new_pinned)
        d.page_copy(s.src, s.dst, s.k, s.v, s.ws)
        return s.new_table, s.new_pinned, s.src, s.dst, s.n_live, s.k, s.v
    d.distill(s.logits, s.ids, s.teacher, s.tau, s.loss, s.ws, grad=s.grad, weight=s.weight, teacher_lse=s.lse)
    return s.loss, s.grad


# ---------------------------------------------------------------------------------------------
# plain forms

def plain_probs(s):
    x = s.logits.float()
    top = x.amax(-1, keepdim=True)
    rate = (LOG2E / s.temperature).clamp(max=1e30)[:, None]
    w = torch.exp2((x - top) * rate)
    p = w / w.sum(-1, keepdim=True)
    first = torch.zeros_like(p).scatter_(-1, (x == top).int().argmax(-1, keepdim=True), 1.0)
    return torch.where((s.temperature <= 0)[:, None], first, p).to(s.probs.dtype)


def _scaled(x, Z):
    """floor(x * Z) for x in [0, 1) on 53 bits and integers Z up to 2^60, exactly."""
    k = (x.double() * 2.0 ** 53).floor().long()
    k1, k0 = k >> 27, k & (2 ** 27 - 1)
    z1, z0 = Z >> 29, Z & (2 ** 29 - 1)
    return k1 * z1 * 8 + ((k1 * z0 + 4 * (k0 * z1) + ((k0 * z0) >> 27)) >> 26)


def plain_verify(s):
    R, G = s.tokens.shape
    start, n = s.q_start[:-1].long(), (s.q_start[1:] - s.q_start[:-1]).long()
    k = torch.arange(G, device=n.device)
    drafted = k < n[:, None] - 1
    at, tok = (start[:, None] + k).clamp(max=s.T - 1), s.tokens.long()
    p = s.target[at, tok].float()
    q = s.draft.gather(-1, tok[..., None])[..., 0].float() if s.draft is not None else torch.ones_like(p)
    ok = (s.u[:, :G] * q.double() < p.double()) & drafted
    a = torch.cumprod(ok.int(), -1).sum(-1)
    rejected = a < n - 1
    P = s.target[start + a].float()
    j = a.clamp(max=G - 1)
    row = torch.arange(R, device=n.device)
    if s.draft is not None:
        Q = s.draft[row, j].float()
    else:
        Q = torch.zeros_like(P).scatter_(-1, tok[row, j][:, None], 1.0)
    Q = torch.where(rejected[:, None], Q, torch.zeros_like(Q))
    mass = lambda w: (w.clamp(0, 1).double() * 2.0 ** 40).long()  # noqa: E731
    fx = mass(P - Q)
    fx = torch.where((fx.sum(-1) > 0)[:, None], fx, mass(P))
    cum = torch.cumsum(fx, -1)
    new = (cum > _scaled(s.u[:, G], cum[:, -1])[:, None]).int().argmax(-1)
    i = torch.arange(G + 1, device=n.device)
    out = torch.cat([tok, tok[:, :1]], -1)
    out = torch.where(i < a[:, None], out, torch.where(i == a[:, None], new[:, None], torch.full_like(out, -1)))
    return out.int(), a.int(), torch.where(drafted, p, torch.zeros_like(p))


def _holders(s):
    need = (s.kv_len + s.page - 1) // s.page
    live = torch.arange(s.width, device=need.device) < need[:, None]
    refs = torch.zeros(s.n_pages + 1, dtype=torch.int32, device=need.device)
    at = torch.where(live, s.table, s.n_pages).flatten().long()
    refs.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    refs.scatter_add_(0, s.pinned.long(), torch.ones_like(s.pinned))
    return refs[:-1], live


def plain_collect(s):
    refs, _ = _holders(s)
    free = torch.argsort((refs > 0).int(), stable=True)
    n = (refs == 0).sum()
    past = torch.arange(s.n_pages, device=refs.device) >= n
    return refs, torch.where(past, torch.full_like(free, -1), free).int(), n.reshape(1).int()


def _copied(s, src, dst, tokens):
    keep = src >= 0
    src, dst, tokens = src[keep].long(), dst[keep].long(), tokens[keep]
    here = torch.arange(s.page, device=src.device) < tokens[:, None]
    for cache in (s.k, s.v):
        for layer in cache:
            layer[dst] = torch.where(here[:, :, None, None], layer[src], layer[dst])


def plain_fork(s):
    n, page = s.parent.numel(), s.page
    length = torch.where(s.parent >= 0, s.length, torch.zeros_like(s.length))
    whole, rest = (length // page).long(), length % page
    col = torch.arange(s.width, device=length.device)
    rows = s.table[s.parent.clamp(min=0).long()]
    table = torch.where(col < (whole + (rest > 0))[:, None], rows, torch.full_like(rows, -1))
    inside = col < whole[:, None]
    held = torch.zeros(s.n_pages + 1, dtype=torch.int32, device=length.device)
    at = torch.where(inside, rows, s.n_pages).flatten().long()
    held.scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    held.scatter_add_(0, s.pinned.long(), torch.ones_like(s.pinned))
    last = rows.gather(1, whole.clamp(max=s.width - 1)[:, None])[:, 0].long()
    last = torch.where(rest > 0, last, s.n_pages)
    row = torch.arange(n, device=length.device)
    first = torch.full_like(held, n).scatter_reduce_(0, last, row.int(), "amin")
    copy = (rest > 0) & ((held[last] > 0) | (first[last] < row))
    new = s.free[(torch.cumsum(copy, 0) - 1).clamp(0, s.free.numel() - 1)]
    none = torch.full_like(new, -1)
    src, dst = torch.where(copy, last.int(), none), torch.where(copy, new, none)
    tokens = torch.where(copy, rest, torch.zeros_like(rest))
    table = torch.where(copy[:, None] & (col == whole[:, None]), new[:, None], table)
    _copied(s, src, dst, tokens)
    return table, length, src, dst, tokens, copy.sum().reshape(1).int(), s.k, s.v


def plain_compact(s):
    refs, inside = _holders(s)
    n = s.n_pages
    live = refs > 0
    m = live.sum()
    page = torch.arange(n, device=refs.device)
    out, into = live & (page >= m), ~live & (page < m)
    pack = lambda keep: torch.full((n + 1,), -1, dtype=torch.int64, device=refs.device).scatter_(  # noqa: E731
        0, torch.where(keep, torch.cumsum(keep, 0) - 1, n), page)[:n // 2]
    src, dst = pack(out), pack(into)
    src[page[:n // 2] >= out.sum()] = -1
    dst[page[:n // 2] >= out.sum()] = -1
    name = torch.cat([page, page[:1]])
    name.scatter_(0, torch.where(src >= 0, src, n), dst)
    table = torch.where(inside, name[s.table.clamp(min=0).long()].int(), torch.full_like(s.table, -1))
    _copied(s, src, dst, torch.full_like(src, s.page))
    return table, name[s.pinned.long()].int(), src.int(), dst.int(), m.reshape(1).int(), s.k, s.v


def plain_distill(s):
    x = s.logits.float() / s.tau
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True, dtype=torch.float64)
    has = s.ids >= 0
    at = s.ids.clamp(min=0).long()
    # the listed entries in 64 bits: what is left of 1, and differences of nearly equal logarithms
    t = s.teacher.double() / s.tau
    if s.lse is None:
        t = t.masked_fill(~has, -math.inf)
        t = t - t.amax(-1, keepdim=True)
        ln_p = t - torch.log(torch.exp(t).sum(-1, keepdim=True))
    else:
        ln_p = t - s.lse.double()[:, None]
    p = torch.where(has, torch.exp(ln_p), torch.zeros_like(t))
    ln_s = s.logits.gather(-1, at).double() / s.tau - top.double() - torch.log(z)
    loss = torch.where(has, p * (ln_p - ln_s), torch.zeros_like(p)).sum(-1)
    share = p.sum(-1, keepdim=True)
    if s.lse is not None:
        out = torch.ones_like(e)
        out.scatter_reduce_(-1, at, (~has).float(), "amin")
        z_rest = (e * out).sum(-1, keepdim=True, dtype=torch.float64)
        p_rest = (1 - share).clamp(min=0)
        some = (p_rest > 0) & (z_rest > 0)
        term = p_rest * (torch.log(p_rest) - torch.log(z_rest) + torch.log(z))
        loss = loss + torch.where(some, term, torch.zeros_like(term))[:, 0]
        share = share + torch.where(some, p_rest, torch.zeros_like(p_rest))
    loss = loss.float()
    if s.grad is None:
        return loss, None
    grad = e * (share / z).float()
    if s.lse is not None:
        grad -= e * out * torch.where(some, p_rest / z_rest, torch.zeros_like(z)).float()
    grad.scatter_add_(-1, at, torch.where(has, -p, torch.zeros_like(p)).float())
    return loss, (grad * (s.weight / s.tau)[:, None]).to(s.logits.dtype)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "probs":
        s = _inputs(case, seed)
        rows = []
        for x, T in zip(s.logits, s.temperature.tolist()):
            y = x.double()
            rows.append(torch.softmax(y / T, 0) if T > 0 else
                        torch.nn.functional.one_hot((y == y.max()).nonzero()[0, 0], len(y)).double())
        return torch.stack(rows)
    if case["op"] == "verify":
        s = _inputs(case, seed)
        p = torch.zeros(s.tokens.shape, dtype=torch.float64, device=s.target.device)
        start = s.q_start.tolist()
        for r in range(p.shape[0]):
            for k in range(start[r + 1] - start[r] - 1):
                p[r, k] = s.target[start[r] + k, s.tokens[r, k]]
        return None, None, p
    if case["op"] == "distill":
        return _exact_distill(_inputs(case, seed))
    return None  # page numbers and copies: nothing is rounded


def _exact_distill(s):
    losses, grads = [], []
    for lo in range(0, len(s.logits), 64):
        at = slice(lo, lo + 64)
        lx = torch.log_softmax(s.logits[at].double() / s.tau, -1)
        N, V = lx.shape
        listed_ids = torch.where(s.ids[at] >= 0, s.ids[at].long(), V)
        t = s.teacher[at].double() / s.tau
        if s.lse is None:
            lp = torch.log_softmax(t.masked_fill(listed_ids == V, -math.inf), -1)
        else:
            lp = (t - s.lse[at].double()[:, None]).masked_fill(listed_ids == V, -math.inf)
        # the teacher as a row over the vocabulary, with one more place for the padding
        full = torch.zeros((N, V + 1), dtype=torch.float64, device=lx.device).scatter_add_(1, listed_ids, lp.exp())[:, :V]
        named = torch.zeros((N, V + 1), dtype=torch.bool, device=lx.device).scatter_(1, listed_ids, True)[:, :V]
        loss = torch.where(named, full * (torch.log(full) - lx), torch.zeros_like(lx)).sum(-1)
        if s.lse is not None:
            rest = (1 - full.sum(-1, keepdim=True)).clamp(min=0)
            tail = torch.where(named, torch.full_like(lx, -math.inf), lx)
            ls_rest = torch.logsumexp(tail, -1, keepdim=True)
            loss = loss + torch.where((rest > 0) & (ls_rest > -math.inf), rest * (torch.log(rest) - ls_rest), 0.0 * rest)[:, 0]
            # a listed entry's target is its own share, the others divide the rest as the student does
            full = full + torch.where(ls_rest > -math.inf, rest * torch.exp(tail - ls_rest), torch.zeros_like(tail))
        losses.append(loss)
        if s.grad is not None:
            grads.append((lx.exp() * full.sum(-1, keepdim=True) - full) * (s.weight[at].double() / s.tau)[:, None])
    return torch.cat(losses), torch.cat(grads) if grads else None
