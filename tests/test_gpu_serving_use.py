"""The serving operators as an engine uses them: on a stream of its own, captured in a graph, over a cache whose
offsets pass 32 bits, in batches whose rows have every kind of sampling parameter."""
import numpy as np
import pytest
import torch

import test_gpu_serving as G
from oracle import serving as S

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark

DEV = "cuda"


def rule_rows(n, seed):
    """Every combination of the four parameters' kinds, a row each in turn."""
    rng = np.random.default_rng(seed)
    i = np.arange(n)
    T = np.where(i % 5 == 4, 0.0, rng.choice([0.6, 1.0, 1.7], n)).astype(np.float32)
    k = np.where(i % 2 == 1, rng.choice([1, 2, 20, 50, 1000], n), 0).astype(np.int32)
    p = np.where(i // 2 % 2 == 1, rng.choice([0.3, 0.9, 0.95, 0.99], n), 1.0).astype(np.float32)
    m = np.where(i // 4 % 2 == 1, rng.choice([0.01, 0.1], n), 0.0).astype(np.float32)
    return T, k, p, m, rng.random(n)


def on_device(rows):
    return tuple(torch.from_numpy(a).to(DEV) for a in rows)


@pytest.mark.parametrize("dtype,N,V,sd", [("bf16", 400, 6001, 1.0), ("bf16", 170, 40000, 2.5), ("fp32", 310, 9000, 2.0)])
def test_many_rows_are_the_rows_alone(dtype, N, V, sd):
    """A row's result does not depend on how many rows the call has or where it stands (which choose the kernel's
    variant), and truncation keeps what sampling draws from."""
    g = torch.Generator().manual_seed(N)
    x = (torch.randn(N, V, generator=g) * sd).to(G.TORCH[dtype]).to(DEV)
    T, k, p, m, u = on_device(rule_rows(N, N))
    ws = G._ws()
    tok, prob = torch.empty(N, dtype=torch.int32, device=DEV), torch.empty(N, device=DEV)
    out = torch.empty_like(x)
    dspark.sample(x, T, k, p, m, u, tok, ws, prob=prob)
    dspark.truncate(x, T, k, p, m, out, ws)
    kept = out > torch.finfo(out.dtype).min
    assert torch.all(kept[torch.arange(N), tok.long()]) and torch.equal(out[kept], x[kept])
    for r in range(0, N, 37):
        t1, p1 = torch.empty(1, dtype=torch.int32, device=DEV), torch.empty(1, device=DEV)
        o1 = torch.empty_like(x[:1])
        s = slice(r, r + 1)
        dspark.sample(x[s], T[s], k[s], p[s], m[s], u[s], t1, ws, prob=p1)
        dspark.truncate(x[s], T[s], k[s], p[s], m[s], o1, ws)
        assert t1.item() == tok[r].item() and p1.item() == prob[r].item() and torch.equal(o1[0], out[r])
    assert dspark.device_status(ws) == dspark.OK


@pytest.mark.parametrize("own_stream", [False, True])
def test_a_step_in_a_graph(own_stream):
    """plan, append, attention, truncation and sampling captured once and replayed with other lengths and values gives
    what the calls give."""
    R, page, Hq, Hkv, D, V, cap = 3, 16, 8, 2, 64, 777, 24
    n_pages = 64  # 30 free ones, eight of each request's own, the prefix's
    rng = np.random.default_rng(1)
    new, cached = torch.zeros(R, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    free = G._i32(rng.permutation(30))
    prefix = G._i32([n_pages - 2, n_pages - 1])
    q, kk, vv = (torch.zeros(cap, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    x = torch.zeros(cap, V, dtype=torch.bfloat16, device=DEV)
    rule = on_device(rule_rows(cap, 2))
    k0, v0 = (torch.randn(n_pages, page, Hkv, D, device=DEV).bfloat16() for _ in range(2))

    def state():
        i32 = dict(dtype=torch.int32, device=DEV)
        return dict(table=torch.arange(30, 30 + 8 * R, **i32).view(R, 8), q_start=torch.zeros(R + 1, **i32), kv_len=torch.zeros(R, **i32),
                    pos=torch.zeros(cap, **i32), slots=torch.zeros(cap, dtype=torch.int64, device=DEV),
                    used=torch.zeros(1, **i32), k=k0.clone(), v=v0.clone(), out=torch.zeros_like(q),
                    lse=torch.zeros(cap, Hq, device=DEV), cut=torch.zeros_like(x), tok=torch.zeros(cap, **i32))

    def step(s, ws, stream=None):
        launches = []
        dspark.page_plan(cached, new, free, page, s["table"], s["q_start"], s["kv_len"], s["pos"], s["slots"], s["used"], ws,
                         stream=stream)
        launches.append(dspark.last_launch_count())
        dspark.kv_append(kk, vv, s["slots"], s["k"], s["v"], ws, stream=stream)
        launches.append(dspark.last_launch_count())
        dspark.prefix_attention(q, s["k"], s["v"], prefix, 20, s["table"], s["q_start"], s["kv_len"], 0.125, s["out"], ws,
                                lse=s["lse"], stream=stream)
        launches.append(dspark.last_launch_count())
        dspark.truncate(x, *rule[:4], s["cut"], ws, stream=stream)
        launches.append(dspark.last_launch_count())
        dspark.sample(x, *rule, s["tok"], ws, stream=stream)
        launches.append(dspark.last_launch_count())
        assert launches == [1, 1, 3, 1, 1]

    ws = dspark.new_attention_workspace(R, cap, Hq, Hkv, D)
    step(state(), ws)  # first-call set-up is done outside the capture
    captured, side = state(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side if own_stream else None):
        step(captured, ws)
    for n, c, seed in (([1, 2, 3], [0, 17, 40], 5), ([8, 8, 8], [16, 0, 99], 6), ([0, 1, 0], [30, 15, 1], 7)):
        new.copy_(torch.tensor(n))
        cached.copy_(torch.tensor(c))
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (q, kk, vv, x):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        fresh = state()
        for name, t in fresh.items():
            captured[name].copy_(t)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        step(fresh, ws)
        assert dspark.device_status(ws) == dspark.OK
        for name in fresh:
            assert torch.equal(fresh[name], captured[name]), name


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, the pages in use at its end (nothing else of it is written or read)."""
    Hq, Hkv, D, page = 8, 8, 128, 64
    c = G.attention_case([3, 1], [150, 70], 200, Hq, Hkv, D, page, seed=8)
    n_small = c["k"].shape[0]
    n_pages = (1 << 32) // (page * Hkv * D) + n_small + 1
    want, want_lse = G.run_attention(c)
    at = n_pages - n_small
    k, v = (torch.empty(n_pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.arange(at * page, n_pages * page, device=DEV)
    ws = G._ws()
    dspark.kv_append(c["k"].view(-1, Hkv, D), c["v"].view(-1, Hkv, D), slots, k, v, ws)
    assert dspark.device_status(ws) == dspark.OK
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731  (NaN past the lengths)
    assert torch.equal(bits(k[at:]), bits(c["k"])) and torch.equal(bits(v[at:]), bits(c["v"]))
    far = dict(c, k=k, v=v, table=c["table"] + at, prefix_pages=c["prefix_pages"] + at)
    out, lse = G.run_attention(far)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("page", [1, 7, 4096, 2 ** 31 - 1])
def test_page_plan_long_lengths(page):
    """Lengths near the end of 32 bits, page sizes that are no power of two."""
    cached, new = [2 ** 31 - 40, 5, 2 ** 30, 0], [33, 0, 17, 9]
    table = np.full((len(cached), 8), 3, dtype=np.int32)
    free = np.arange(100, 100 + 64)
    got = G.run_plan(cached, new, free, page, table, 64)
    G.check_plan(got, S.page_plan(cached, new, free, page, table, 64))


def test_page_plan_sum_past_31_bits():
    """A request whose length would pass 2^31 - 1 is reported and held at it; the others are right."""
    t, q_start, kv_len, pos, slots, used, status = G.run_plan([2 ** 31 - 3, 4], [9, 2], np.arange(4), 4096, np.zeros((2, 4), np.int32), 11)
    assert status in (dspark.ERR_RANGE, dspark.ERR_CAPACITY)
    assert q_start.tolist() == [0, 9, 11] and kv_len.tolist() == [2 ** 31 - 1, 6]
    assert pos.tolist()[9:] == [4, 5] and slots.tolist()[9:] == [4, 5]


def plain_rule(x, T, k, p, m, u):
    """The rule's definition with torch's operations on the device, row by row: kept mask and token. The same float32
    weights (CUDA's exp2f on the same argument), masses and sums in integers."""
    V = x.numel()
    x = x.float()
    M = x.max()
    rate = min(np.float32(np.float32(1.4426950408889634) / np.float32(T)), np.float32(1e30))
    mass = (torch.exp2((x - M) * float(rate)).double() * 2.0 ** 40).floor().long()
    order = torch.sort(x, descending=True, stable=True).indices
    sorted_mass = mass[order]
    n = V if k <= 0 or k >= V else k
    before = sorted_mass.cumsum(0) - sorted_mass
    if p < 1:
        S = int(sorted_mass[:n].sum())
        num, den = float(p).as_integer_ratio()
        n = min(n, int((before[:n] < max(1, S * num // den)).sum()))
    kept = torch.zeros(V, dtype=torch.bool, device=x.device)
    kept[order[:n]] = True
    kept &= mass >= 0 if m <= 0 else torch.exp2((x - M) * float(rate)) >= float(np.float32(m))
    kept &= x > -float("inf")
    mass = torch.where(kept, mass, 0)
    c = mass.cumsum(0)
    num, den = float(u).as_integer_ratio()
    return kept, int((c > int(c[-1]) * num // den).nonzero()[0])


def shaped_row(kind, V, rng):
    x = rng.normal(size=V) * 2
    if kind == "descending":
        x = -np.sort(-x)
    elif kind == "ascending":
        x = np.sort(x)
    elif kind == "one_above":      # one entry far above all others, late in the row
        x[V - 3] = 60.0
    elif kind == "some_above":     # a few hundred, of differing weights, above what the row's start shows
        x[-V // 5:][::37] += 20 + rng.random(len(x[-V // 5:][::37])) * 12
    elif kind == "two_levels":     # half the row far below the other half
        x[rng.permutation(V)[:V // 2]] -= 45
    elif kind == "ramp":           # hundreds of octaves from end to end
        x = np.linspace(-300, 20, V)[rng.permutation(V)]
    elif kind == "wide":
        x *= 40
    return x.astype(np.float32)


KINDS = ["normal", "descending", "ascending", "one_above", "some_above", "two_levels", "ramp", "wide"]


@pytest.mark.parametrize("dtype,V", [("bf16", 6001), ("bf16", 65537), ("fp32", 30011), ("bf16", 129280), ("fp32", 600000)])
def test_rule_on_shaped_rows(dtype, V):
    """Rows whose distribution over values and over indices differs from what a row's start or a sample of it
    shows: exactly the definition's kept set and token, in both kernels."""
    rng = np.random.default_rng(V)
    rows = [(kind, T, k, p, m) for kind in KINDS
            for T, k, p, m in [(1.0, 0, 0.95, 0.0), (1.7, 0, 0.9, 0.0), (1.3, 0, 0.999, 1e-5), (0.2, 0, 0.99, 0.0), (1.0, 1000, 1.0, 0.0),
                               (1.5, 3000, 0.9, 0.0), (0.6, 7, 0.8, 0.1), (2.0, 0, 1.0, 0.02)]]
    x = torch.from_numpy(np.stack([shaped_row(kind, V, rng) for kind, *_ in rows])).to(DEV).to(G.TORCH[dtype])
    T, k, p, m = (np.array(a) for a in list(zip(*rows))[1:])
    u = rng.random(len(rows))
    for n in (len(rows), 200):  # alone on its SM, and with other rows
        g = np.arange(n) % len(rows)
        tokens, prob, out, st, st2 = G.run_rule(x[torch.from_numpy(g).to(DEV)].contiguous(), T[g], k[g], p[g], m[g], u[g])
        assert st == dspark.OK and st2 == dspark.OK
        for i in range(len(rows)):
            kept, token = plain_rule(x[i], np.float32(T[i]), int(k[i]), np.float32(p[i]), m[i], u[i])
            G.check_kept(x, out[i:i + 1].repeat(i + 1, axis=0), i, kept.cpu().numpy())
            assert tokens[i] == token, rows[i]
        if n == 200 and V > 200000:
            break


def test_rule_at_infinite_temperature():
    """Temperature inf: every finite entry weighs 1, whatever its size."""
    x = torch.tensor([[-3e38, 3e38, 0.0, -float("inf"), 1.0, 2.0]], device=DEV).repeat(3, 1)
    tokens, prob, out, st, _ = G.run_rule(x, np.float32(np.inf), 0, 1.0, 0.0, [0.05, 0.5, 0.99])
    assert st == dspark.OK and set(tokens.tolist()) <= {0, 1, 2, 4, 5}
