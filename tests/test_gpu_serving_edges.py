"""Serving operators where one call's result meets another's assumptions: short token capacities, calls without
tokens, scores that are no number, temperatures and logits at the ends of float32."""
import math

import numpy as np
import pytest
import torch

import test_gpu_serving as G
import test_gpu_serving_use as U
from oracle import serving as S

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# a plan whose token capacity runs out

@pytest.mark.parametrize("capacity", [0, 1, 4, 7, 8, 11, 300, 301, 1000, "128 requests", "256 requests"])
@pytest.mark.parametrize("page", [1, 16])
def test_page_plan_past_its_capacity(capacity, page):
    """A short plan is the plan of the tokens that fit, with the status word set: lengths, table entries and pages taken
    as if the request that is cut had asked for what is left of it, and the later ones for nothing."""
    rng = np.random.default_rng(5)
    R = 400
    c, n = rng.integers(0, 50, R), rng.integers(0, 6, R)
    n[:3] = [4, 3, 4]
    if isinstance(capacity, str):  # exactly what the first of them ask for
        capacity = int(n[:int(capacity.split()[0])].sum())
    width = int((-(-(c + n) // page)).max())
    table = np.arange(R * width).reshape(R, width)
    free = 100000 + rng.permutation(3000)
    fit = np.clip(capacity - (np.cumsum(n) - n), 0, n)
    want = S.page_plan(c, fit, free, page, table, capacity)
    t, q_start, kv_len, pos, slots, used, status = G.run_plan(c, n, free, page, table, capacity)
    assert status == (dspark.ERR_CAPACITY if n.sum() > capacity else dspark.OK)
    assert q_start.tolist() == want["q_start"] and kv_len.tolist() == want["kv_len"]
    assert np.array_equal(t.cpu().numpy(), want["table"]) and used.item() == want["used"]
    assert pos.tolist() == want["positions"] and slots.tolist() == want["slots"]


def test_attention_after_a_short_plan():
    """plan -> append -> attention with room for 6 of 9 new tokens: the tokens that fit are attended at their own
    positions, over keys that were appended (the others' slots hold NaN)."""
    page, Hq, Hkv, D = 16, 4, 2, 64
    cached, new, capacity = [20, 15, 40], [3, 4, 2], 6
    whole = G.attention_case([3, 3], [23, 18], 0, Hq, Hkv, D, page, seed=11)  # request 1 cut to 3 tokens, request 2 without
    n_pages = whole["k"].shape[0] + 4
    k, v = (torch.full((n_pages, page, Hkv, D), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kn, vn = (torch.full((sum(new), Hkv, D), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.full((3, 4), n_pages - 1, dtype=torch.int32, device=DEV)
    free, at = [], 0
    for r in range(2):
        for j in range(-(-int(whole["kv_len"][r]) // page)):
            src, first = int(whole["table"][r, j]), j * page
            if first < cached[r]:
                table[r, j] = src
                m = min(page, cached[r] - first)
                k[src, :m], v[src, :m] = whole["k"][src, :m], whole["v"][src, :m]
            else:
                free.append(src)
        for i in range(3):
            pos = cached[r] + i
            pg, off = int(whole["table"][r, pos // page]), pos % page
            kn[at], vn[at] = whole["k"][pg, off], whole["v"][pg, off]
            at += 1
    free += list(range(whole["k"].shape[0], n_pages - 1))
    i32 = dict(dtype=torch.int32, device=DEV)
    q_start, kv_len, pos = torch.empty(4, **i32), torch.empty(3, **i32), torch.empty(capacity, **i32)
    slots, used = torch.empty(capacity, dtype=torch.int64, device=DEV), torch.empty(1, **i32)
    ws = G._ws()
    dspark.page_plan(G._i32(cached), G._i32(new), G._i32(free), page, table, q_start, kv_len, pos, slots, used, ws)
    assert dspark.device_status(ws) == dspark.ERR_CAPACITY
    dspark.kv_append(kn[:capacity], vn[:capacity], slots, k, v, G._ws())
    want, want_lse = G.run_attention(whole)
    got, got_lse = G.run_attention(dict(whole, k=k, v=v, table=table, q_start=q_start, kv_len=kv_len))
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


# ---------------------------------------------------------------------------------------------
# a call without tokens

def test_attention_without_tokens():
    c = G.attention_case([0, 0], [40, 8], 64, 8, 2, 64, 16)
    assert c["q"].shape[0] == 0
    out, lse = G.run_attention(c)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    out, _ = G.run_attention(G.attention_case([0, 0], [40, 8], 64, 8, 2, 64, 16, capacity=3))
    assert torch.all(out == 77.0)


# ---------------------------------------------------------------------------------------------
# scores that are no number

@pytest.mark.parametrize("private,prefix", [(9, 0), (700, 0), (9, 3000), (300, 40)])
def test_attention_of_a_nan_query(private, prefix):
    """A query that holds a NaN has no softmax: NaN, however many parts its keys are split into, and in its row alone."""
    c = G.attention_case([3, 1], [private, 50], prefix, 8, 2, 64, 16, seed=12)
    want, want_lse = G.run_attention(c)
    c["q"][1, 5, 3] = math.nan
    out, lse = G.run_attention(c)
    assert torch.all(torch.isnan(out[1, 5])) and torch.isnan(lse[1, 5])
    out[1, 5], lse[1, 5] = want[1, 5], want_lse[1, 5]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


# ---------------------------------------------------------------------------------------------
# sampling: temperatures and logits at the ends of float32

def test_rule_at_infinite_temperature_is_uniform():
    """Every finite entry weighs 1, whatever its size and whatever the distance to the maximum overflows to."""
    inf = math.inf
    x = torch.tensor([[-3e38, 3e38, 0.0, -inf, 1.0, 2.0]], device=DEV).repeat(6, 1)
    tokens, prob, out, st, _ = G.run_rule(x, np.float32(np.inf), [0, 0, 0, 0, 4, 0], [1.0, 1.0, 1.0, 0.5, 1.0, 1.0],
                                          [0.0, 0.0, 0.0, 0.0, 0.0, 1.0], [0.05, 0.5, 0.99, 0.99, 0.99, 0.99])
    assert st == dspark.OK
    # kept: all five; by logit 3e38, 2, 1 reach a mass of 2.5 of 5; the four largest; all five reach min_p = 1
    assert tokens.tolist() == [0, 2, 5, 5, 5, 5]
    assert np.allclose(prob, [0.2, 0.2, 0.2, 1 / 3, 0.25, 0.2], rtol=2.0 ** -22)
    low = float(torch.finfo(torch.float32).min)
    assert np.array_equal(out[0] == low, [False, False, False, True, False, False])
    assert np.array_equal(out[3] == low, [True, False, True, True, False, False])
    assert np.array_equal(out[4] == low, [True, False, False, True, False, False])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [3e35, 2e36, 3e37, 1e38, 3.4e38, np.inf])
@pytest.mark.parametrize("V,at", [(3, 0), (90, 0), (90, 1), (5000, 3)])
def test_rule_at_huge_temperatures(dtype, T, V, at):
    """Logits of up to float32's range at temperatures of the same size, against the oracle in 64 bits. (The rate is
    rounded to float32 or below its normal range, 2^-149 of up to 2^-126.8 at 3.4e38: 2^-22, times an exponent of at most 6.)"""
    rng = np.random.default_rng([V, at])
    x = (rng.random((24, V)) * 6.7e38 - 3.35e38).astype(np.float32)
    x[::4, ::3] = -math.inf
    x[:, V // 2] = 3.3e38
    flat = torch.zeros(24 * V + at, dtype=G.TORCH[dtype], device=DEV)
    xt = flat[at:].view(24, V)
    xt.copy_(torch.from_numpy(x))
    k, p = rng.choice([0, 0, 2, V // 2], 24), rng.choice([1.0, 1.0, 0.4, 0.9], 24).astype(np.float32)
    m, u = rng.choice([0.0, 0.0, 0.2], 24).astype(np.float32), rng.random(24)
    tokens, prob, out, st, st2 = G.run_rule(xt, np.float32(T), k, p, m, u)
    assert st == dspark.OK and st2 == dspark.OK
    eps, sure = 2.0 ** -17 + V * 2.0 ** -40, 0
    for r in range(24):
        kept, w, margin = S.rule(xt[r].float().cpu().numpy(), float(np.float32(T)), int(k[r]), float(p[r]), float(m[r]))
        if margin <= 4 * eps:
            continue
        G.check_kept(xt, out, r, kept)
        v, pr, gap = S.draw(kept, w, u[r])
        if gap <= 4 * eps:
            continue
        sure += 1
        assert tokens[r] == v and abs(prob[r] - pr) <= 4 * eps * pr + 2.0 ** -40
    assert sure >= 8


# ---------------------------------------------------------------------------------------------
# sampling: a search for top-p's end that moves its range across zero

@pytest.mark.parametrize("rows", [1, 200])
def test_top_p_ranges_that_meet_at_zero(rows):
    """A row whose sampled distribution (the largest and the first entry of four) misleads the search for top-p's end
    twice, each time further down, with the second range ending at a logit of 0 that hundreds of entries have. At the
    temperature whose rate is 1, with bins of 1/64:
      first   of the estimate's mass the limit lies at logit 1 and the next bin with entries is that of 2/64
      second  from 1.5/64 down; 1/64 is estimated at four times its number, so that the range goes no further than 0
      third   from 0 down, exclusive: the limit is met among the entries of -1/64
    Weights 2^(x - 1), the masses in floor(. 2^40): kept set and token in exact integers."""
    T = np.float32(1.4426950408889634)
    rng = np.random.default_rng(4)
    r = -0.05
    pieces = ([[1 / 64, 1.0, r, r]] * 1525 + [[1.0, r, r, r]] * 2000 + [[2 / 64, r, r, r]] * 20 + [[-1 / 64, r, r, r]] * 100)
    x = np.array(pieces, dtype=np.float32)[rng.permutation(len(pieces))]
    hidden = np.flatnonzero(x[:, 0] > 0)  # where the third of four is neither the first nor the largest
    x[rng.permutation(hidden)[:400], 2] = 0.0
    x = x.reshape(-1)
    w = np.floor(np.exp2(x.astype(np.float64) - 1) * 2.0 ** 40)
    ten = 10 * 2.0 ** 40  # of the 49.5 that the entries of -1/64 weigh
    p = np.float32((w[x >= 0].sum() + ten) / w.sum())
    xt = torch.from_numpy(np.tile(x, (rows, 1))).to(DEV)
    tokens, prob, out, st, _ = G.run_rule(xt, T, 0, p, 0.0, np.linspace(0.0, 0.999, rows))
    assert st == dspark.OK
    kept, _ = (a.cpu().numpy() if torch.is_tensor(a) else a for a in U.plain_rule(xt[0], T, 0, p, 0.0, 0.5))
    assert kept[x >= 0].all() and 15 <= kept[x < 0].sum() <= 25 and np.all(x[kept] >= np.float32(-1 / 64))
    for i in range(rows):
        G.check_kept(xt, out, i, kept)
    c = np.cumsum(np.where(kept, w, 0.0))
    for i, u in enumerate(np.linspace(0.0, 0.999, rows)):
        assert tokens[i] == np.searchsorted(c, u * c[-1], side="right") or np.abs(c - u * c[-1]).min() < 2.0 ** -17 * c[-1]


# ---------------------------------------------------------------------------------------------
# sampling: one weight for an entry, whichever part of a call forms it

@pytest.mark.parametrize("dtype,V", [("fp32", 8), ("fp32", 4100), ("bf16", 16)])
def test_every_token_has_the_mass_it_is_drawn_by(dtype, V):
    """Rows over many exponents at the temperature whose rate is 1 (maximum 0: the exponent is the logit), drawn at a
    uniform in the middle of one entry's mass: that token, with its mass over the row's, masses floor(2^x 2^40) by
    torch's float32 exp2. Entries next to the drawn one are as large, so that a unit's difference between the sum and the
    walk would show."""
    N = (1 << 21) // V
    g = torch.Generator(device=DEV).manual_seed(V)
    x = -40 * torch.rand((N, V), generator=g, device=DEV) ** 2
    x[:, 0] = 0.0
    x = x.to(G.TORCH[dtype])
    mass = (torch.exp2(x.float()).double() * 2.0 ** 40).floor().long()
    c = mass.cumsum(1)
    at = torch.randint(0, V, (N,), generator=g, device=DEV)
    here, Z = mass.gather(1, at[:, None])[:, 0], c[:, -1]
    first = c.gather(1, at[:, None])[:, 0] - here
    u = (first.double() + 0.5 * here.double()) / Z.double()
    sure = here > (Z >> 51) + 8  # (u is rounded to 2^-53 of 1)
    par = (torch.full((N,), 1.4426950408889634, device=DEV), torch.zeros(N, dtype=torch.int32, device=DEV),
           torch.ones(N, device=DEV), torch.zeros(N, device=DEV))
    tokens, prob, ws = torch.full((N,), -7, dtype=torch.int32, device=DEV), torch.full((N,), -7.0, device=DEV), G._ws()
    dspark.sample(x, *par, u, tokens, ws, prob=prob)
    assert dspark.device_status(ws) == dspark.OK
    assert torch.equal(tokens[sure].long(), at[sure]) and int(sure.sum()) > N // 2
    want = (here.double() / Z.double()).float()
    assert torch.equal(prob[sure], want[sure])


# ---------------------------------------------------------------------------------------------
# rows of several temperatures for a verification at one

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_other_temperatures_scale_to_one(dtype):
    """Rows of temperature T_r, multiplied by T / T_r and truncated at T, keep what they keep at T_r; at ratios of two
    every step of the weights is the same float32 number."""
    rng = np.random.default_rng(21)
    T, ratio = 0.8, np.tile([0.5, 1.0, 2.0, 4.0], 10).astype(np.float32)
    x = torch.from_numpy((rng.normal(size=(40, 5000)) * 2).astype(np.float32)).to(DEV).to(G.TORCH[dtype])
    f = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DEV)  # noqa: E731
    k, p, m = G._i32(rng.choice([0, 20, 400], 40)), f(rng.choice([0.9, 0.99, 1.0], 40)), f(rng.choice([0.0, 0.01], 40))
    scaled = (x.float() * f(ratio)[:, None]).to(x.dtype)
    a, b, ws = torch.empty_like(x), torch.empty_like(x), G._ws()
    dspark.truncate(x, f(np.float32(T) / ratio), k, p, m, a, ws)
    dspark.truncate(scaled, f(np.full(40, T)), k, p, m, b, ws)
    low = torch.finfo(x.dtype).min
    assert dspark.device_status(ws) == dspark.OK and torch.equal(a > low, b > low) and not torch.all(a > low)


# ---------------------------------------------------------------------------------------------
# plans of more requests than a block has threads, long pages, long prompts

@pytest.mark.parametrize("new,private,prefix,Hq,Hkv,D,page", [
    ([i % 3 for i in range(1500)], [2 + (i * 37) % 90 for i in range(1500)], 70, 2, 1, 64, 16),   # two turns of the plan
    ([1] * 2049, [1 + i % 40 for i in range(2049)], 0, 2, 2, 64, 32),                             # three, the last one request
    ([2, 1] * 5 + [0] * 1100 + [3], [300 + i for i in range(10)] + [5] * 1100 + [200], 150, 4, 1, 128, 16),
    ([3, 1], [1500, 700], 1000, 4, 2, 128, 512),                                                  # a page of several tiles
    ([2], [5000], 4097, 4, 1, 64, 4096),                                                          # the longest page
    ([1100, 1], [1300, 40], 200, 2, 1, 64, 16),                                                   # a prompt chunk of many blocks
])
def test_attention_of_many_requests_and_long_ones(new, private, prefix, Hq, Hkv, D, page):
    c = G.attention_case(new, private, prefix, Hq, Hkv, D, page)
    G.check_attention(c, *G.run_attention(c))
