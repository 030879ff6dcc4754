"""GPU parity of the serving operators (page plan, KV append, shared-prefix attention, sampling rule)
with the float64 oracle.

Integers are compared for equality. Attention: out is rounded to bf16 once (half a step of an 8-bit
significand, 2^-8 relative), its weights to bf16 before the product with v (2^-8 of sum_j w_j |v_j|), the two
exponential evaluations and float32 sums stay under 2^-18 of it, and a score error e scales each
weight by at most 1 + 2 e. lse carries the score error and float32 roundings of its own size.
Sampling: a weight's exponent has two float32 roundings at magnitude up to 40 and exp2f two units,
so masses are within 2^-17 relative and V 2^-40 absolute of the real ones: rows whose nearest
comparison is further than that must agree exactly."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import serving as S

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark

DEV = "cuda"


def _ws():
    return dspark.new_workspace(1, 1, 1, 1, dspark.FP32, 1)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


# ---------------------------------------------------------------------------------------------
# pages and slots

def run_plan(cached, new, free, page, table, capacity):
    R = len(cached)
    t = _i32(table)
    q_start, kv_len = torch.full((R + 1,), -7, dtype=torch.int32, device=DEV), torch.full((R,), -7, dtype=torch.int32, device=DEV)
    pos = torch.full((capacity,), -7, dtype=torch.int32, device=DEV)
    slots = torch.full((capacity,), -7, dtype=torch.int64, device=DEV)
    used = torch.full((1,), -7, dtype=torch.int32, device=DEV)
    ws = _ws()
    dspark.page_plan(_i32(cached), _i32(new), _i32(free), page, t, q_start, kv_len, pos, slots, used, ws)
    return t, q_start, kv_len, pos, slots, used, dspark.device_status(ws)


def check_plan(got, want):
    t, q_start, kv_len, pos, slots, used, status = got
    assert np.array_equal(t.cpu().numpy(), want["table"])
    assert q_start.tolist() == want["q_start"] and kv_len.tolist() == want["kv_len"]
    assert pos.tolist() == want["positions"] and slots.tolist() == want["slots"] and used.item() == want["used"]
    assert status == (dspark.ERR_CAPACITY if want["short"] else dspark.OK)


@pytest.mark.parametrize("R,new,cached,page,spare", [
    (1, 1, 0, 16, 0), (1, 0, 5, 16, 0), (3, 17, 40, 1, 3), (127, 9, 300, 64, 5), (128, 17, 100, 16, 0),
    (129, 17, 64, 16, 1), (700, 33, 50, 24, 0), (2049, 3, 10, 128, 2)])
def test_page_plan(R, new, cached, page, spare):
    rng = np.random.default_rng(R + page)
    c, n = rng.integers(0, cached + 1, R), rng.integers(0, new + 1, R)
    have, need = -(-c // page), -(-(c + n) // page)
    width = int(max(need.max(), 1)) + spare
    ids = rng.permutation(int(need.sum()) + 3)
    table = np.full((R, width), 7, dtype=np.int32)
    held = np.arange(width) < have[:, None]
    table[held] = ids[:held.sum()]
    free = ids[held.sum():]
    capacity = int(n.sum()) + spare
    check_plan(run_plan(c, n, free, page, table, capacity), S.page_plan(c, n, free, page, table, capacity))


def test_page_plan_runs_out():
    """Pages, table columns and token capacity that run out: -1 entries, nothing outside the tensors."""
    rng = np.random.default_rng(3)
    R, page = 300, 16
    c, n = rng.integers(0, 64, R), rng.integers(0, 40, R)
    for width, n_free, capacity in [(8, 100, int(n.sum())), (4, 2000, int(n.sum())), (8, 2000, 1000), (8, 0, 5000), (5, 50, 0)]:
        table = np.full((R, width), 3, dtype=np.int32)
        free = rng.permutation(n_free)
        check_plan(run_plan(c, n, free, page, table, capacity), S.page_plan(c, n, free, page, table, capacity))


def test_page_plan_negative_length():
    got = run_plan([4, -1, 2], [1, 3, -5], [8, 9], 4, [[1], [0], [2]], 4)
    assert got[-1] == dspark.ERR_RANGE or got[-1] == dspark.ERR_CAPACITY
    assert got[2].tolist() == [5, 3, 2] and got[1].tolist() == [0, 1, 4, 4]


# ---------------------------------------------------------------------------------------------
# append

@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,Hkv,D,n_slots", [(0, 8, 128, 16), (1, 1, 64, 16), (37, 3, 5, 64), (1153, 8, 128, 2048), (300, 2, 64, 1 << 16)])
def test_kv_append(dtype, T, Hkv, D, n_slots):
    dt = getattr(torch, dtype)
    g = torch.Generator(device=DEV).manual_seed(T)
    k, v = (torch.randn((T, Hkv, D), generator=g, device=DEV).to(dt) for _ in range(2))
    kc, vc = (torch.randn((n_slots // 16, 16, Hkv, D), generator=g, device=DEV).to(dt) for _ in range(2))
    slots = torch.randperm(n_slots, generator=g, device=DEV)[:T].contiguous()
    slots[::7] = -1
    want_k, want_v = kc.clone().view(n_slots, Hkv, D), vc.clone().view(n_slots, Hkv, D)
    live = slots >= 0
    want_k[slots[live]], want_v[slots[live]] = k[live], v[live]
    ws = _ws()
    dspark.kv_append(k, v, slots, kc, vc, ws)
    assert dspark.device_status(ws) == dspark.OK
    assert torch.equal(kc.view_as(want_k), want_k) and torch.equal(vc.view_as(want_v), want_v)


def test_kv_append_slot_out_of_range():
    k = torch.ones((3, 1, 8), dtype=torch.float32, device=DEV)
    kc = torch.zeros((1, 16, 1, 8), dtype=torch.float32, device=DEV)
    vc = kc.clone()
    ws = _ws()
    dspark.kv_append(k, k, torch.tensor([2, 16, 1 << 40], device=DEV), kc, vc, ws)
    assert dspark.device_status(ws) == dspark.ERR_RANGE
    assert kc.sum().item() == 8 and vc[0, 2].sum().item() == 8


def test_kv_append_unaligned_rows():
    """A view that starts 2 bytes into its storage, and rows of 10 bytes."""
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(41 * 5 + 1, generator=g, device=DEV).bfloat16()[1:].view(41, 1, 5)
    kc, vc = torch.zeros((4, 16, 1, 5), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 16, 1, 5), dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(63, 22, -1, device=DEV)
    ws = _ws()
    dspark.kv_append(k, k, slots, kc, vc, ws)
    assert torch.equal(kc.view(64, 1, 5)[slots], k) and torch.equal(vc.view(64, 1, 5)[slots], k)


# ---------------------------------------------------------------------------------------------
# attention

def attention_case(new, private, prefix, Hq, Hkv, D, page, seed=0, spare_pages=2, q_scale=1.0, capacity=None):
    """Inputs whose cache holds NaN past every length, with a shuffled page order."""
    rng = np.random.default_rng([seed, prefix, Hq, D, page])
    R, T = len(new), int(sum(new))
    cap = T if capacity is None else capacity
    need = [-(-x // page) for x in private]
    npre = -(-prefix // page)
    n_pages = sum(need) + npre + spare_pages
    ids = rng.permutation(n_pages)
    k = np.full((n_pages, page, Hkv, D), np.nan, dtype=np.float32)
    v = k.copy()
    width = max(max(need), 1) + 1
    table = np.full((R, width), n_pages - 1, dtype=np.int32)
    def fill(pages, length):
        for j, pg in enumerate(pages):
            m = min(page, length - j * page)
            k[pg, :m], v[pg, :m] = rng.normal(size=(2, m, Hkv, D))

    pre, at = ids[:npre], npre
    fill(pre, prefix)
    for r in range(R):
        table[r, :need[r]] = ids[at:at + need[r]]
        fill(table[r, :need[r]], private[r])
        at += need[r]
    q = rng.normal(size=(cap, Hq, D)) * q_scale
    bf = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV).bfloat16()  # noqa: E731
    return dict(q=bf(q), k=bf(k), v=bf(v), prefix_pages=_i32(pre), prefix_len=prefix, table=_i32(table),
                q_start=_i32(np.concatenate([[0], np.cumsum(new)])), kv_len=_i32(private), scale=1.0 / math.sqrt(D))


def run_attention(c, ws=None, want=dspark.OK if torch.cuda.is_available() else 0, stream=None):
    T, Hq, D = c["q"].shape
    out = torch.full_like(c["q"], 77.0)
    lse = torch.full((T, Hq), 77.0, device=DEV)
    if ws is None:
        ws = dspark.new_attention_workspace(c["kv_len"].numel(), T, Hq, c["k"].shape[2], D)
    dspark.prefix_attention(c["q"], c["k"], c["v"], c["prefix_pages"], c["prefix_len"], c["table"], c["q_start"],
                            c["kv_len"], c["scale"], out, ws, lse=lse, stream=stream)
    assert dspark.device_status(ws, stream) == want
    return out, lse


def check_attention(c, out, lse):
    n = lambda t: t.float().cpu().numpy()  # noqa: E731
    T = int(c["q_start"][-1])
    ref, ref_lse, spread, err = S.attention(n(c["q"])[:T], n(c["k"]), n(c["v"]), c["prefix_pages"].cpu().numpy(), c["prefix_len"],
                                            c["table"].cpu().numpy(), c["q_start"].tolist(), c["kv_len"].tolist(), c["scale"])
    got, got_lse = n(out)[:T], n(lse)[:T].astype(np.float64)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -18 + 2 * err[..., None]) * spread * (1 + 2.0 ** -8) + 1e-30
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) / bound))
    empty = np.isneginf(ref_lse)
    assert np.all(np.isneginf(got_lse[empty])) and not got[empty].any()
    far = np.abs(got_lse[~empty] - ref_lse[~empty])
    assert np.all(far <= err[~empty] + 2.0 ** -19 * (1 + np.abs(ref_lse[~empty])))
    # rows past the last query are left alone
    assert torch.all(out[T:] == 77.0) and torch.all(lse[T:] == 77.0)


SHAPES = [
    # new, private, prefix, Hq, Hkv, D, page
    ([1], [1], 0, 1, 1, 64, 16),                        # one key
    ([1], [1], 1, 8, 8, 128, 16),                       # one key in each part
    ([1], [333], 1000, 32, 8, 128, 64),
    ([3], [3], 0, 4, 2, 128, 64),                       # a causal triangle alone
    ([17], [17], 15, 12, 4, 64, 16),                    # the prefix ends inside the first page
    ([5, 0, 1, 9], [130, 40, 128, 9], 129, 16, 2, 128, 32),   # ragged, an idle request, one key past a tile
    ([40, 70], [300, 70], 500, 28, 4, 64, 16),          # 7 heads a key head: rows do not fill a tile
    ([33], [200], 77, 5, 1, 128, 128),                  # 5 heads a key head
    ([2, 1], [700, 90], 640, 128, 1, 64, 64),           # 128 heads on one key head
    ([4] * 9, [257] * 9, 2000, 24, 8, 128, 256),        # pages longer than a tile
    ([1] * 40, list(range(1, 41)), 31, 8, 4, 64, 16),
    ([300], [300], 0, 4, 1, 128, 16),                   # a prompt chunk: causal over three tiles
    ([6, 4], [3, 0], 0, 6, 3, 64, 16),                  # more queries than keys: empty rows, then a request with none
    ([6, 4], [3, 0], 5, 6, 3, 128, 16),                 # the same with a prefix
    ([2, 2], [4500, 9], 9000, 8, 2, 64, 16),            # long: split over keys
    # many more items than SMs, of one to five tiles, a half's rows and two halves' in turn
    ([1 + i % 3 for i in range(220)], [3 + (i * 37) % 620 for i in range(220)], 300, 32, 8, 64, 16),
    ([1 + (i * 7) % 40 for i in range(90)], [41 + (i * 53) % 500 for i in range(90)], 130, 16, 4, 128, 32),
]


@pytest.mark.parametrize("new,private,prefix,Hq,Hkv,D,page", SHAPES)
def test_attention(new, private, prefix, Hq, Hkv, D, page):
    c = attention_case(new, private, prefix, Hq, Hkv, D, page)
    check_attention(c, *run_attention(c))


@pytest.mark.parametrize("q_scale", [0.0, 30.0])
def test_attention_flat_and_sharp(q_scale):
    """Equal scores, and scores whose running maximum jumps by far more than float32's exponent range of weights."""
    c = attention_case([9, 2], [250, 31], 400, 8, 2, 128, 32, seed=4, q_scale=q_scale)
    check_attention(c, *run_attention(c))


def test_attention_query_capacity():
    """Query rows past q_start[R] (a batch padded to a fixed size) are left alone."""
    c = attention_case([3, 1], [40, 8], 64, 8, 2, 64, 16, capacity=11)
    check_attention(c, *run_attention(c))


def test_attention_repeats_bit_for_bit():
    c = attention_case([9, 1, 17], [900, 300, 170], 3000, 16, 4, 128, 64, seed=5)
    T, Hq, D = c["q"].shape
    ws = dspark.new_attention_workspace(3, T, Hq, 4, D)
    out, lse = run_attention(c, ws)
    for _ in range(20):
        o, z = run_attention(c, ws)
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_attention_on_another_stream_without_lse():
    c = attention_case([5], [90], 200, 8, 2, 128, 64, seed=6)
    want, _ = run_attention(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    T, Hq, D = c["q"].shape
    out = torch.zeros_like(c["q"])
    ws = dspark.new_attention_workspace(1, T, Hq, 2, D, stream=s)
    dspark.prefix_attention(c["q"], c["k"], c["v"], c["prefix_pages"], c["prefix_len"], c["table"], c["q_start"], c["kv_len"],
                            c["scale"], out, ws, stream=s)
    assert dspark.device_status(ws, s) == dspark.OK and torch.equal(out, want)


def test_attention_bad_tables():
    """A page id outside the cache, a length past the table and a falling q_start are reported; nothing outside the
    tensors is read and the other requests' rows are right."""
    good = attention_case([2, 2], [40, 50], 70, 8, 2, 64, 16, seed=7)
    want, _ = run_attention(good)
    for field, at, value in [("table", (0, 1), 10 ** 6), ("table", (0, 0), -5), ("kv_len", (0,), 10 ** 7), ("kv_len", (0,), -3)]:
        c = dict(good)
        c[field] = good[field].clone()
        c[field][at] = value
        out, _ = run_attention(c, want=dspark.ERR_RANGE)
        assert torch.equal(out[2:], want[2:])
    c = dict(good, q_start=_i32([0, 10 ** 6, 4]))
    run_attention(c, want=dspark.ERR_RANGE)
    c = dict(good, q_start=_i32([-9, 2, 4]))
    run_attention(c, want=dspark.ERR_RANGE)


def test_attention_refusals():
    c = attention_case([2], [40], 20, 8, 2, 64, 16)
    ws = dspark.new_attention_workspace(1, 2, 8, 2, 64)
    call = lambda **kw: run_attention({**c, **kw}, ws)  # noqa: E731
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(dspark.DSparkError) as e:
            call(**kw)
        assert e.value.status == dspark.ERR_INVALID_ARG
    for bad in (c["k"][:, :12].contiguous(), c["k"].view(-1, 16, 1, 128)[:, :, :, :32].contiguous()):  # a page of 12; head_dim 32
        with pytest.raises((dspark.DSparkError, ValueError)):
            call(k=bad, v=bad)
    with pytest.raises(ValueError, match="contiguous"):
        call(k=c["k"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        call(prefix_len=c["prefix_pages"].numel() * 16 + 1)
    with pytest.raises(TypeError):
        call(q=c["q"].float(), k=c["k"].float(), v=c["v"].float())
    odd = torch.zeros(2 * 8 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(2, 8, 64)
    with pytest.raises(dspark.DSparkError):
        call(q=odd)
    with pytest.raises(dspark.DSparkError) as e:
        run_attention(c, ws[:dspark.attention_workspace_bytes(1, 2, 8, 2, 64) - 256])
    assert e.value.status == dspark.ERR_WORKSPACE


# ---------------------------------------------------------------------------------------------
# the sampling rule

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}


def run_rule(x, temperature, top_k, top_p, min_p, u):
    """x on the device; tokens, prob, truncated rows (as numpy) and both status words."""
    N = x.shape[0]
    f = lambda a, dt: torch.from_numpy(np.array(np.broadcast_to(a, N), dtype=dt)).to(DEV)  # noqa: E731
    par = (f(temperature, np.float32), f(top_k, np.int32), f(top_p, np.float32), f(min_p, np.float32))
    tokens = torch.full((N,), -7, dtype=torch.int32, device=DEV)
    prob = torch.full((N,), -7.0, device=DEV)
    ws, ws2 = _ws(), _ws()
    dspark.sample(x, *par, f(u, np.float64), tokens, ws, prob=prob)
    out = torch.full_like(x, 7.0)
    dspark.truncate(x, *par, out, ws2)
    inplace = x.clone()
    dspark.truncate(inplace, *par, inplace, ws2)
    assert torch.equal(inplace.view(torch.uint8), out.view(torch.uint8))
    return tokens.cpu().numpy(), prob.cpu().numpy().astype(np.float64), out.float().cpu().numpy(), dspark.device_status(ws), dspark.device_status(ws2)


def check_kept(x, out, r, kept):
    lowest = float(torch.finfo(x.dtype).min)
    row = x[r].float().cpu().numpy()
    assert np.array_equal(out[r], np.where(kept, row, np.float32(lowest)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,sd", [(1, 1, 1.0), (40, 7, 2.0), (30, 1000, 2.0), (24, 4099, 4.0), (16, 32003, 1.5), (6, 129280, 2.0), (3, 300000, 3.0)])
def test_rule_matches_oracle(dtype, N, V, sd):
    rng = np.random.default_rng([N, V])
    x = torch.from_numpy((rng.normal(size=(N, V)) * sd - 1.1 * np.log1p(rng.permutation(V))).astype(np.float32)).to(DEV).to(TORCH[dtype])
    T = rng.choice([0.0, 0.3, 0.7, 1.0, 1.5], N).astype(np.float32)
    k = rng.choice([0, 1, 5, 50, 1000, V, V + 5], N)
    p = rng.choice([1.0, 0.5, 0.9, 0.99, 0.0], N).astype(np.float32)
    m = rng.choice([0.0, 0.0, 0.05, 0.3], N).astype(np.float32)
    u = rng.random(N)
    tokens, prob, out, st, st2 = run_rule(x, T, k, p, m, u)
    assert st == dspark.OK and st2 == dspark.OK
    eps = 2.0 ** -17 + V * 2.0 ** -40
    sure = 0
    for r in range(N):
        kept, w, margin = S.rule(x[r].float().cpu().numpy(), float(T[r]), int(k[r]), float(p[r]), float(m[r]))
        if margin <= 4 * eps:
            continue
        check_kept(x, out, r, kept)
        v, pr, gap = S.draw(kept, w, u[r])
        if gap <= 4 * eps:
            continue
        sure += 1
        assert tokens[r] == v
        assert abs(prob[r] - pr) <= 4 * eps * pr + 2.0 ** -40
    assert sure >= N // 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [1, 2, 31, 64, 1000, 4096, 5003, 40000, 131072])
def test_rule_exact_on_powers_of_two(dtype, V):
    """Whole logits at the temperature whose rate is 1: every mass is a power of two, so the kept set, its ties
    and the drawn token follow in exact integers. Few distinct values: every threshold falls among ties."""
    rng = np.random.default_rng(V)
    T = np.float32(1.4426950408889634)
    N = 24
    x = -rng.integers(0, 6, (N, V)).astype(np.float32) - rng.integers(0, 2, (N, 1)) * 3
    x[::5] -= rng.integers(0, 50, (len(x[::5]), V))  # weights down to 2^-50: masses of 0
    x[3] = 0.0                                        # constant rows
    x[7] = -3.0
    x[11, :-1] = -np.inf                              # one live entry
    x[12, ::2] = -np.inf
    x[12, -1] = 0.0
    x[13] = -0.0
    x[13, ::3] = 0.0                                  # both zeros are one value
    k = rng.choice([0, 1, 2, 7, V // 2, V - 1], N)
    p = rng.choice([1.0, 0.25, 0.5, 0.75, 0.999], N).astype(np.float32)
    m = rng.choice([0.0, 0.0, 0.125, 0.5], N).astype(np.float32)
    u = np.concatenate([[0.0, 1 - 2.0 ** -53], rng.integers(0, 16, 6) / 16, rng.random(N - 8)])
    xt = torch.from_numpy(x).to(DEV).to(TORCH[dtype])
    tokens, prob, out, st, st2 = run_rule(xt, T, k, p, m, u)
    assert st == dspark.OK and st2 == dspark.OK
    for r in range(N):
        kept, v, pr = S.exact_rule(x[r].astype(np.float64).tolist(), 1.0, int(k[r]), float(p[r]), float(m[r]), u[r])
        mask = np.zeros(V, dtype=bool)
        mask[kept] = True
        check_kept(xt, out, r, mask)
        assert tokens[r] == v and abs(prob[r] - pr) <= 2.0 ** -23 * pr


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rule_masked_and_extreme_rows(dtype):
    """Entries at the type's lowest value and at -inf, tiny and huge temperatures, u at and past its ends."""
    V = 700
    lowest = float(torch.finfo(TORCH[dtype]).min)
    x = torch.full((6, V), lowest, device=DEV, dtype=TORCH[dtype])
    x[0, 300:310] = 2.0                # ten live entries in a masked row
    x[1] = lowest                      # everything at the lowest value: uniform
    x[2, 5] = -float("inf")
    x[3, 600] = 1e30
    x[4, 17], x[4, 18] = 3.0, 2.0
    x[5] = torch.linspace(-1, 1, V, device=DEV).to(TORCH[dtype])
    T = [1.0, 1.0, 1.0, 1.0, 1e-38, 1e30]
    tokens, prob, out, st, _ = run_rule(x, T, 0, 1.0, 0.0, [0.95, 0.5, 0.0, 0.3, 0.999, 1.0])
    assert st == dspark.OK
    assert tokens.tolist()[:5] == [309, 350, 0, 600, 17] and tokens[5] == V - 1
    assert np.allclose(prob, [0.1, 1 / V, 1 / (V - 1), 1.0, 1.0, 1 / V], rtol=1e-6)
    assert out[2, 5] == lowest


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rule_rows_without_a_distribution(dtype):
    x = torch.zeros((4, 50), device=DEV, dtype=TORCH[dtype])
    x[0, 3], x[1, 9], x[2] = float("nan"), float("inf"), -float("inf")
    x[3, 8] = 1.0
    tokens, prob, out, st, st2 = run_rule(x, [1.0, 0.0, 1.0, 0.0], 5, 0.9, 0.0, 0.5)
    assert st == dspark.ERR_NONFINITE and st2 == dspark.ERR_NONFINITE
    assert tokens.tolist() == [-1, -1, -1, 8] and prob.tolist() == [0, 0, 0, 1]
    assert np.array_equal(out[:3], x[:3].float().cpu().numpy(), equal_nan=True)


def test_rule_unaligned_rows():
    """Odd row lengths and a first element that is not 16-byte aligned."""
    rng = np.random.default_rng(9)
    flat = torch.from_numpy(rng.normal(size=5 * 4097 + 3).astype(np.float32)).to(DEV)
    for dt in (torch.bfloat16, torch.float32):
        base = flat.to(dt)
        for off in (0, 1, 3):
            x = base[off:off + 5 * 4097].view(5, 4097)
            tokens, prob, out, st, _ = run_rule(x, 0.9, 40, 0.95, 0.0, rng.random(5))
            assert st == dspark.OK
            for r in range(5):
                kept, _, margin = S.rule(x[r].float().cpu().numpy(), float(np.float32(0.9)), 40, float(np.float32(0.95)), 0.0)
                if margin > 2.0 ** -15:
                    check_kept(x, out, r, kept)


def test_rule_refusals():
    x = torch.zeros((2, 8), device=DEV)
    f = torch.ones(2, device=DEV)
    k = torch.zeros(2, dtype=torch.int32, device=DEV)
    u, t, ws = torch.zeros(2, dtype=torch.float64, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV), _ws()
    with pytest.raises(TypeError):
        dspark.sample(x, f, k, f, f, u.float(), t, ws)
    with pytest.raises(ValueError):
        dspark.sample(x, f[:1], k, f, f, u, t, ws)
    with pytest.raises(TypeError):
        dspark.truncate(x.half(), f, k, f, f, x.half(), ws)
    with pytest.raises(dspark.DSparkError) as e:
        dspark.sample(x, f, k, f, f, u, t, ws[:128])
    assert e.value.status == dspark.ERR_WORKSPACE
    with pytest.raises(dspark.DSparkError):
        big = torch.zeros((1, (1 << 20) + 1), device=DEV)
        dspark.truncate(big, f[:1], k[:1], f[:1], f[:1], big, ws)
