"""GPU parity of the calls after the target's pass with the float64 oracle.

Integers (tokens, lengths, page ids) and copies are compared for equality. Probabilities and gradients: the
exponent of a weight 2^y has its difference, its product and its rate rounded (4 roundings of 2^-24 of |y|, ln 2 of
that in the weight), ex2.approx is within 2^-22 of the power, a sum of weights carries its terms' errors and
at most 45 roundings (64 terms a thread in two chains, a tree over the cluster), and the scaling three. Results are rounded
once more to their type: half a step, 2^-8 of the value in bf16. Weights below 2^-126 are 0."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import target_pass as O

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark

DEV = "cuda"
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DTYPES = [torch.float32, torch.bfloat16]


def ws_small():
    return dspark.new_workspace(1, 1, 1, 1, dspark.FP32, 1)


def on(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def i32(a):
    return on(np.asarray(a, dtype=np.int32), torch.int32)


def blank(*shape, dtype=torch.int32):
    return torch.full(shape, -7, dtype=dtype, device=DEV)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def weight_error(octaves, mean_octaves):
    """Relative error of a weight of 2^-octaves over the sum of all, in float32."""
    return 4 * math.log(2) * 2.0 ** -24 * (octaves + mean_octaves) + 2 * 2.0 ** -22 + 48 * 2.0 ** -24


# ---------------------------------------------------------------------------------------------
# probabilities

def check_probs(x, T, out, status=None):
    ws = ws_small()
    probs = torch.full(x.shape, -7.0, dtype=out, device=DEV)
    dspark.probabilities(x, on(np.asarray(T, dtype=np.float32), torch.float32), probs, ws)
    assert dspark.device_status(ws) == (status or dspark.OK)
    rows, got = host(x), host(probs)
    for r in range(len(rows)):
        p, y = O.softmax(rows[r], np.float64(np.float32(T[r])))
        if not p.any() or not T[r] > 0:
            assert np.array_equal(got[r], p), r
            continue
        bound = p * (weight_error(np.abs(y), (p * np.abs(y)).sum()) + HALF_STEP[out]) + 2.0 ** -125
        assert (np.abs(got[r] - p) <= bound).all(), (r, np.max(np.abs(got[r] - p) / bound))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (2, 7), (5, 17), (1, 1000), (4, 4097), (3, 32003), (300, 2050), (2, 129280)])
def test_probabilities(dtype, out, N, V):
    rng = np.random.default_rng(N * V)
    x = on(rng.normal(size=(N, V)) * 3, dtype)
    check_probs(x, rng.choice([0.0, 0.3, 1.0, 1.7, 40.0], N), out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V", [(3, 262151), (2, 1 << 20)])
def test_probabilities_of_long_rows(dtype, N, V):
    """Rows that no cluster holds: read again."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn((N, V), generator=g, device=DEV) * 2).to(dtype)
    check_probs(x, [0.8, 0.0, 1.3][:N], torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_probabilities_of_masked_and_extreme_rows(dtype):
    lowest = torch.finfo(dtype).min
    rows = np.zeros((9, 40))
    rows[0, 3:] = -math.inf                # three entries left
    rows[1, :] = -math.inf
    rows[1, 39] = 2.0                      # one
    rows[2, 5:] = float(lowest)            # as truncated rows come
    rows[3] = np.arange(40) * 1e30         # far apart
    rows[4] = np.arange(40)
    rows[5] = np.arange(40) * 1e4
    rows[6] = 7.0                          # all equal
    rows[7, ::2] = -math.inf
    rows[8] = np.linspace(-3e38, 3e38, 40) # past float32's range apart
    x = on(rows, torch.float64).to(dtype)
    T = [1.0, 0.5, 1.0, 1.0, 1e-38, 1e-4, 2.0, math.inf, 1e38]
    check_probs(x, T, torch.float32)
    check_probs(x, [0.0] * 8 + [-1.0], torch.float32)


def test_probabilities_of_bad_rows():
    for bad in (math.nan, math.inf):
        x = torch.zeros((3, 5000), device=DEV)
        x[1, 4321] = bad
        check_probs(x, [1.0, 1.0, 0.0], torch.float32, status=dspark.ERR_NONFINITE)
    x = torch.full((2, 50), -math.inf, device=DEV)
    check_probs(x, [1.0, 0.0], torch.float32, status=dspark.ERR_NONFINITE)


@pytest.mark.parametrize("dtype", DTYPES)
def test_probabilities_unaligned(dtype):
    """Rows of a tensor that does not begin at a 16-byte boundary, results neither, on other offsets."""
    rng = np.random.default_rng(4)
    base = on(rng.normal(size=5 * 1003 + 8), dtype)
    for a, b in [(1, 0), (0, 1), (3, 3), (5, 2)]:
        x = base[a:a + 5 * 1003].view(5, 1003)
        whole = torch.full((5 * 1003 + 8,), -7.0, device=DEV)
        probs = whole[b:b + 5 * 1003].view(5, 1003)
        ws = ws_small()
        dspark.probabilities(x, torch.full((5,), 0.9, device=DEV), probs, ws)
        for r in range(5):
            p, y = O.softmax(host(x)[r], np.float64(np.float32(0.9)))
            assert (np.abs(host(probs)[r] - p) <= p * weight_error(np.abs(y), (p * np.abs(y)).sum()) + 2.0 ** -125).all()
        assert (whole[:b] == -7).all() and (whole[b + 5 * 1003:] == -7).all()


# ---------------------------------------------------------------------------------------------
# verification

def run_verify(target, q_start, draft, tokens, u):
    R, gamma = tokens.shape
    out, acc, p_tok = blank(R, gamma + 1), blank(R), blank(R, gamma, dtype=torch.float32)
    ws = ws_small()
    dspark.verify_probs(target, i32(q_start), draft, i32(tokens), on(u, torch.float64), out, acc, p_tok, ws)
    return out.cpu().numpy(), acc.cpu().numpy(), p_tok.cpu().numpy(), dspark.device_status(ws)


def check_verify(target, q_start, draft, tokens, u, status=0):
    want = O.verify_probs(target.float().cpu().numpy(), q_start, None if draft is None else draft.float().cpu().numpy(), tokens, u)
    got = run_verify(target, q_start, draft, tokens, u)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)
    assert got[3] == status
    return got


def block(seed, R, gamma, V, dtype, sharp=3.0, near=0.5):
    rng = np.random.default_rng(seed)
    n = rng.integers(0, gamma + 2, R)
    n[0] = gamma + 1
    q_start = np.concatenate([[0], np.cumsum(n)])
    x = rng.normal(size=(R, gamma + 1, V)) * sharp
    soft = lambda a: np.exp(a - a.max(-1, keepdims=True)) / np.exp(a - a.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    P, Q = soft(x), soft(x[:, :gamma] + near * rng.normal(size=(R, gamma, V)))
    target = on(np.concatenate([P[r, :n[r]] for r in range(R)]), torch.float32).to(dtype)
    draft = on(Q, torch.float32).to(dtype)
    tokens = np.array([[rng.choice(V, p=Q[r, k] / Q[r, k].sum()) for k in range(gamma)] for r in range(R)])
    return target, q_start, draft, tokens, rng.random((R, gamma + 1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,gamma,V", [(1, 1, 1), (1, 1, 2), (3, 4, 7), (7, 16, 130), (40, 5, 1000), (3, 33, 64), (2, 70, 33),
                                     (5, 3, 32003), (2, 2, 129280), (200, 2, 97)])
def test_verify_probs(dtype, R, gamma, V):
    b = block(R * V, R, gamma, V, dtype)
    check_verify(*b)
    check_verify(b[0], b[1], None, *b[3:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_verify_probs_at_the_longest_row(dtype):
    V = 1 << 20
    g = torch.Generator(device=DEV).manual_seed(2)
    P = torch.softmax(torch.randn((3, V), generator=g, device=DEV), -1).to(dtype)
    Q = torch.softmax(torch.randn((1, 2, V), generator=g, device=DEV), -1).to(dtype)
    for u in (0.0, 0.5, 1 - 2.0 ** -53):
        check_verify(P, [0, 3], Q, np.array([[V - 1, 5]]), np.array([[u, u, u]]))
    # every entry at the largest mass: the sum is 2^60
    P = torch.ones((1, V), device=DEV, dtype=dtype)
    for u in (0.0, 0.3, 1 - 2.0 ** -53):
        check_verify(P, [0, 1], None, np.array([[0]]), np.array([[0.5, u]]))


def test_verify_probs_draws_at_the_edges():
    """Uniforms at a mass's first and last step, masses far apart, the only entry with mass at either end of the row."""
    V = 5000
    P = torch.zeros((4, V), device=DEV)
    P[0, 0], P[1, V - 1], P[2, 17], P[2, 4000] = 1.0, 1.0, 2.0 ** -40, 2.0 ** -41  # 2^-41 has no mass
    P[3] = 1.0 / 4096
    for u in (0.0, 2.0 ** -53, 0.25, 0.25 - 2.0 ** -53, 0.5, 1 - 2.0 ** -53):
        tokens = np.array([[3]] * 4)
        check_verify(P, [0, 1, 2, 3, 4], None, tokens, np.array([[0.5, u]] * 4))


def test_verify_probs_boundaries_of_acceptance():
    """u q = p is a rejection, the next smaller uniform an acceptance; q = 0 stands iff p > 0."""
    P = torch.tensor([[0.25, 0.75], [0.5, 0.5], [0.0, 1.0], [0.5, 0.5], [0.25, 0.75], [0.5, 0.5], [0.25, 0.75], [0.5, 0.5]], device=DEV)
    Q = torch.tensor([[[0.5, 0.5]], [[0.0, 1.0]], [[0.0, 1.0]], [[0.5, 0.5]]], device=DEV)
    u = np.array([[0.5, 0.1], [0.9, 0.1], [0.9, 0.1], [0.5 - 2.0 ** -53, 0.1]])
    got = check_verify(P, [0, 2, 4, 6, 8], Q, np.array([[0]] * 4), u)
    assert got[1].tolist() == [0, 0, 1, 1]


def test_verify_probs_bad_inputs():
    P = torch.full((4, 6), 1 / 6, device=DEV)
    tokens, u = np.array([[1, 2]] * 2), np.full((2, 3), 0.5)
    check_verify(P, [0, 2, 4], None, np.array([[6, 2], [-1, 2]]), u, status=dspark.ERR_RANGE)
    for q_start in ([0, 2, 5], [-1, 2, 4], [0, 3, 2]):
        check_verify(P, q_start, None, tokens, u, status=dspark.ERR_RANGE)
    check_verify(P, [0, 4, 4], None, tokens, u, status=dspark.ERR_RANGE)  # three drafts where two have room
    check_verify(P, [0, 0, 0], None, tokens, u)
    for bad in (math.nan, math.inf):
        Pb = P.clone()
        Pb[0, 3] = bad
        check_verify(Pb, [0, 1, 2], None, tokens, u, status=dspark.ERR_NONFINITE)
    check_verify(P * 0, [0, 2, 4], None, tokens, u, status=dspark.ERR_NONFINITE)
    # no row at all
    out = run_verify(torch.empty((0, 6), device=DEV), [0, 0, 0], None, tokens, u)
    assert (out[0] == -1).all() and not out[1].any() and out[3] == dspark.OK


def test_verify_probs_unaligned():
    V = 1001
    target, q_start, draft, tokens, u = block(5, 6, 3, V, torch.bfloat16)
    for a, b in [(1, 0), (0, 3), (5, 5)]:
        t = torch.cat([target.new_zeros(a), target.flatten()])[a:].view_as(target)
        q = torch.cat([draft.new_zeros(b), draft.flatten()])[b:].view_as(draft)
        check_verify(t, q_start, q, tokens, u)


# ---------------------------------------------------------------------------------------------
# pages

def table_of(rng, R, width, page, n_pages, share=0):
    """Rows over distinct random pages, the first `share` full pages of row 0 in every row."""
    ids = rng.permutation(n_pages)
    kv_len = rng.integers(0, width * page + 1, R)
    kv_len[rng.integers(0, R)] = width * page
    table, at = rng.integers(-5, n_pages + 5, (R, width)), 0  # anything past a row's length
    for r in range(R):
        n = -(-kv_len[r] // page)
        s = min(n, share, kv_len[0] // page) if r else 0
        if at + n - s > n_pages:
            kv_len[r] = 0
            continue
        table[r, :s], table[r, s:n] = table[0, :s], ids[at:at + n - s]
        at += n - s
    return table, kv_len, ids[at:]


SHAPES = [(1, 1, 16, 1, 0), (1, 3, 1, 9, 0), (4, 5, 16, 40, 2), (130, 9, 64, 1500, 4), (1100, 3, 16, 4000, 0), (3, 700, 16, 2500, 300),
          (2000, 40, 16, 90000, 10), (20000, 6, 32, 70001, 2)]


def run_collect(table, kv_len, page, n_pages, pinned):
    refs, free, n = blank(n_pages), blank(n_pages), blank(1)
    ws = dspark.new_page_workspace(n_pages)
    dspark.page_collect(i32(table), i32(kv_len), page, refs, free, n, ws, pinned=i32(pinned) if len(pinned) else None)
    return refs, free, n, dspark.device_status(ws)


@pytest.mark.parametrize("R,width,page,n_pages,share", SHAPES)
def test_page_collect(R, width, page, n_pages, share):
    rng = np.random.default_rng(R + width)
    table, kv_len, spare = table_of(rng, R, width, page, n_pages, share)
    for pinned in ([], [int(x) for x in spare[:5]], [int(table[kv_len.argmax(), 0])] * 2):
        refs, free, n, status = run_collect(table, kv_len, page, n_pages, pinned)
        want = O.page_collect(table, kv_len, page, n_pages, pinned)
        assert refs.tolist() == want[0] and free.tolist() == want[1] and n.item() == want[2] and status == dspark.OK


def run_fork(table, kv_len, parent, length, page, n_pages, free, pinned):
    n, width = len(parent), table.shape[1]
    got = {"new_table": blank(n, width), "new_len": blank(n), "src": blank(n), "dst": blank(n), "tokens": blank(n), "used": blank(1)}
    ws = dspark.new_page_workspace(n_pages)
    dspark.page_fork(i32(table), i32(kv_len), i32(parent), None if length is None else i32(length), page, n_pages, i32(free), *got.values(),
                     ws, pinned=i32(pinned) if len(pinned) else None)
    return {k: v.tolist() for k, v in got.items()} | {"used": got["used"].item()}, dspark.device_status(ws)


@pytest.mark.parametrize("R,width,page,n_pages,share", SHAPES)
def test_page_fork(R, width, page, n_pages, share):
    rng = np.random.default_rng(R * 3 + width)
    table, kv_len, spare = table_of(rng, R, width, page, n_pages, share)
    pinned = [int(x) for x in spare[:2]] + [int(table[kv_len.argmax(), -1])]
    free = spare[2:]
    for n, cut in [(R, False), (max(1, R // 2), True), (R + R // 3 + 1, True)]:
        parent = rng.integers(-1, R, n) if cut else rng.permutation(R)
        length = np.array([0 if q < 0 else rng.integers(0, kv_len[q] + 1) for q in parent]) if cut else None
        want = O.page_fork(table, kv_len, parent, length, page, n_pages, free, pinned)
        got, status = run_fork(table, kv_len, parent, length, page, n_pages, free, pinned)
        assert got == want
        short = any(row[-(-m // page) - 1] < 0 for row, m in zip(want["new_table"], want["new_len"]) if m)
        assert status == (dspark.ERR_CAPACITY if short else dspark.OK)


def test_page_fork_rows_cut_inside_shared_pages():
    """Rows that end inside one page: the first keeps it, unless it is another's full page or pinned."""
    table, kv_len = np.array([[4, 2, 9], [4, 7, -1]]), [12, 7]
    for parent, length, pinned in [([0, 0, 0], [6, 7, 5], []), ([0, 0], [6, 12], []), ([1, 0, 1], [2, 3, 7], []), ([0], [6], [2]),
                                   ([0, 1, -1, 0], [12, 4, 0, 4], [])]:
        want = O.page_fork(table, kv_len, parent, length, 4, 10, [0, 1, 3], pinned)
        assert run_fork(table, kv_len, parent, length, 4, 10, [0, 1, 3], pinned) == (want, dspark.OK)


def test_page_fork_bad_inputs():
    table, kv_len = np.array([[4, 2], [30, -1]]), [6, 3]
    for parent, length, free, status in [([0, 0], [5, 6], [], dspark.ERR_CAPACITY), ([0, 0, 0], [5, 6, 5], [1, -1, -1], dspark.ERR_CAPACITY),
                                         ([2, -2, 0], [5, 6, 5], [1], dspark.ERR_RANGE), ([0], [7], [1], dspark.ERR_RANGE),
                                         ([0], [-1], [1], dspark.ERR_RANGE), ([1, 1], [3, 3], [1], dspark.ERR_RANGE)]:
        want = O.page_fork(table, kv_len, parent, length, 4, 10, free, [])
        got = run_fork(table, kv_len, parent, length, 4, 10, free, [])
        assert got == (want, status)


@pytest.mark.parametrize("R,width,page,n_pages,share", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_page_compact(R, width, page, n_pages, share, in_place):
    rng = np.random.default_rng(R * 5 + width)
    table, kv_len, spare = table_of(rng, R, width, page, n_pages, share)
    pinned = [int(x) for x in spare[:3]]
    t, pin = i32(table), i32(pinned)
    new_table, new_pinned = (t, pin) if in_place else (blank(R, width), blank(len(pinned)))
    src, dst, n_live = blank(n_pages // 2), blank(n_pages // 2), blank(1)
    ws = dspark.new_page_workspace(n_pages)
    dspark.page_compact(t, i32(kv_len), page, n_pages, new_table, src, dst, n_live, ws, pinned=pin if pinned else None,
                        new_pinned=new_pinned)
    want = O.page_compact(table, kv_len, page, n_pages, pinned)
    got = {"new_table": new_table.tolist(), "new_pinned": new_pinned.tolist(), "src": src.tolist(), "dst": dst.tolist(),
           "n_live": n_live.item()}
    assert got == want and dspark.device_status(ws) == dspark.OK


def test_page_calls_report_bad_tables():
    """Ids outside the cache and lengths past the table: reported, left out, carried along."""
    table, kv_len = np.array([[3, 99], [-1, 2], [0, 1]]), [8, 8, 9]
    refs, free, n, status = run_collect(table, kv_len, 4, 6, [])
    assert status == dspark.ERR_RANGE and refs.tolist() == O.page_collect(table, kv_len, 4, 6)[0] and n.item() == 2
    new, src, dst, n_live = blank(3, 2), blank(3), blank(3), blank(1)
    ws = dspark.new_page_workspace(6)
    dspark.page_compact(i32(table), i32(kv_len), 4, 6, new, src, dst, n_live, ws)
    assert dspark.device_status(ws) == dspark.ERR_RANGE and new.tolist() == [[3, 99], [-1, 2], [0, 1]] and n_live.item() == 4
    refs, _, n, status = run_collect(table[2:], [-3], 4, 6, [7, 5])
    assert status == dspark.ERR_RANGE and refs.tolist() == [0, 0, 0, 0, 0, 1] and n.item() == 5


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layers,n_pages,page,Hkv,D", [(1, 4, 16, 1, 8), (2, 40, 16, 2, 64), (3, 30, 64, 8, 128), (1, 9, 3, 3, 5), (2, 6, 4096, 1, 64)])
def test_page_copy(dtype, layers, n_pages, page, Hkv, D):
    g = torch.Generator(device=DEV).manual_seed(page)
    k, v = (torch.randn((layers, n_pages, page, Hkv, D), generator=g, device=DEV).to(dtype) for _ in range(2))
    rng = np.random.default_rng(page)
    ids = rng.permutation(n_pages)
    n = n_pages // 2
    src, dst = ids[:n].copy(), ids[n:2 * n].copy()
    src[::5] = -1
    tokens = rng.integers(-2, page + 3, n)
    for use in (tokens, None):
        want = [c.clone() for c in (k, v)]
        for a, b, m in zip(src, dst, tokens if use is not None else [page] * n):
            if a >= 0:
                for c in want:
                    c[:, b, :max(m, 0)] = c[:, a, :max(m, 0)]
        ws = ws_small()
        dspark.page_copy(i32(src), i32(dst), k, v, ws, tokens=None if use is None else i32(tokens))
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and dspark.device_status(ws) == dspark.OK
    ws = ws_small()
    dspark.page_copy(i32([0, n_pages]), i32([n_pages, 0]), k, v, ws)
    assert torch.equal(k, want[0]) and dspark.device_status(ws) == dspark.ERR_RANGE


# ---------------------------------------------------------------------------------------------
# distillation

def run_distill(x, ids, t, tau, lse=None, weight=None, back=True, in_place=False):
    N = x.shape[0]
    loss = torch.full((N,), -7.0, device=DEV)
    grad = (x if in_place else torch.full_like(x, -7.0)) if back else None
    ws = ws_small()
    f32 = lambda a: None if a is None else on(np.asarray(a, dtype=np.float32), torch.float32)  # noqa: E731
    dspark.distill(x, i32(ids), f32(t), tau, loss, ws, grad=grad, weight=f32(weight), teacher_lse=f32(lse))
    return host(loss), None if grad is None else host(grad), dspark.device_status(ws)


def check_distill(x, ids, t, tau, lse=None, weight=None, **kw):
    """tau and all float32 inputs are taken as the values they are. A logarithm of s has its weight's error; the rate's
    rounding scales a distance from the maximum by 2^-23 at most."""
    rows = host(x)
    loss, grad, status = run_distill(x, ids, t, tau, lse, weight, **kw)
    dt = x.dtype
    for r in range(len(rows)):
        L, G, parts = O.distill(rows[r], ids[r], np.asarray(t, dtype=np.float32)[r], tau, None if lse is None else np.float32(lse[r]))
        s, p, below = parts["s"], parts["p"], parts["below"]
        mean_s, mean_p = (s * below).sum(), (p * np.where(p > 0, below, 0)).sum()
        e_z = weight_error(0.0, mean_s / math.log(2))
        e_rest = weight_error(0.0, (s[~parts["named"]] * below[~parts["named"]]).sum() / math.log(2) / max(parts["s_rest"], 1e-300))
        total = p.sum() + parts["p_rest"]
        if math.isfinite(L):
            bound = 2.0 ** -22 * (mean_p + mean_s) + e_z * total + parts["p_rest"] * e_rest + 2.0 ** -23 * abs(L) + 1e-30
            assert abs(loss[r] - L) <= bound, (r, loss[r], L, bound)
        else:
            assert loss[r] == L or math.isnan(loss[r]) and math.isnan(L)
            if math.isnan(L):
                assert grad is None or not grad[r].any()
                continue
        if grad is None:
            continue
        w = 1.0 if weight is None else float(np.float32(weight[r]))
        e_s = weight_error(below / math.log(2), mean_s / math.log(2))
        share = parts["p_rest"] / parts["s_rest"] if parts["p_rest"] > 0 else 0.0
        bound = (s * total * e_s + np.where(parts["named"], p * 2.0 ** -23, s * share * (e_s + e_rest))) * abs(w) / tau
        bound += HALF_STEP[dt] * np.abs(G * w) * (1 + 2.0 ** -8) + 2.0 ** -125
        err = np.abs(grad[r] - G * w)
        assert (err <= bound * (1 + HALF_STEP[dt])).all(), (r, np.max(err / bound), int(np.argmax(err / bound)))
    return loss, grad, status


def problem(seed, N, V, K, dtype, tau, near=0.5):
    rng = np.random.default_rng(seed)
    full = rng.normal(size=(N, V)) * 3
    x = on(full + near * rng.normal(size=(N, V)), dtype)
    ids = np.argsort(-full, axis=1, kind="stable")[:, :K]
    t = np.take_along_axis(full, ids, 1)
    top = full.max(1)
    lse = top / tau + np.log(np.exp((full - top[:, None]) / tau).sum(1))
    return x, ids, t, lse, rng


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("N,V,K,tau", [(1, 1, 1, 1.0), (2, 2, 2, 1.0), (3, 9, 4, 0.5), (5, 130, 1, 2.0), (200, 1001, 20, 1.0), (4, 32003, 64, 1.5),
                                       (2, 5000, 1024, 1.0), (3, 129280, 64, 1.0), (700, 64, 8, 4.0)])
def test_distill(dtype, rest, N, V, K, tau):
    x, ids, t, lse, rng = problem(N + V, N, V, K, dtype, tau)
    weight = rng.normal(size=N)
    weight[::3] = 0
    loss, grad, status = check_distill(x, ids, t, tau, lse if rest else None, weight)
    assert status == dspark.OK and not grad[::3].any()
    # the loss alone, and the gradient over the logits, are the same bits
    alone = run_distill(x, ids, t, tau, lse if rest else None, back=False)
    over = run_distill(x.clone(), ids, t, tau, lse if rest else None, weight, in_place=True)
    assert np.array_equal(alone[0], loss) and np.array_equal(over[0], loss) and np.array_equal(over[1], grad)


@pytest.mark.parametrize("dtype", DTYPES)
def test_distill_long_rows(dtype):
    """Rows that no cluster holds: read again, and overwritten in place."""
    for V in (262160, 1 << 20):
        x, ids, t, lse, _ = problem(V, 2, V, 30, dtype, 1.0)
        ids[0, 0], ids[1, 1] = V - 1, 0
        loss, grad, _ = check_distill(x, ids, t, 1.0, lse)
        over = run_distill(x.clone(), ids, t, 1.0, lse, in_place=True)
        assert np.array_equal(over[0], loss) and np.array_equal(over[1], grad)


@pytest.mark.parametrize("rest", [False, True])
def test_distill_lists(rest):
    """Padded and empty lists, an id that comes twice or thrice, ids out of range, listed entries at the row's ends."""
    V, K = 1003, 6
    x, ids, t, lse, _ = problem(1, 8, V, K, torch.float32, 1.5)
    ids[0, 3:] = -1
    ids[1] = -1
    ids[2, :] = ids[2, 0]
    ids[3, 4] = ids[3, 1]
    ids[4] = [0, V - 1, 1, V - 2, 2, V - 3]
    ids[5, :] = [-1, 7, -1, 7, -5, 8]
    lse = lse + 1.0  # the teacher's rest has mass for every list
    assert check_distill(x, ids, t, 1.5, lse if rest else None)[2] == dspark.OK
    ids[6, 2] = V
    assert check_distill(x, ids, t, 1.5, lse if rest else None)[2] == dspark.ERR_RANGE


def test_distill_masked_and_extreme_rows():
    inf, V = math.inf, 300
    x = torch.zeros((7, V), device=DEV)
    x[0, 10:] = -inf                                  # a masked drafter, listed entries inside
    x[1, 10:] = torch.finfo(torch.float32).min
    x[2] = torch.arange(V, device=DEV) * 100.0        # one entry has all the mass
    x[3] = torch.linspace(-3e38, 3e38, V, device=DEV)  # its step overflows: a row with NaN
    x[6] = torch.linspace(-3e38, 3e38, V, dtype=torch.float64).float()  # distances past float32's range
    x[4, 5] = -inf                                    # a listed entry without probability
    ids = np.tile(np.arange(4), (7, 1))
    ids[2], ids[3], ids[4], ids[6] = [299, 298, 297, 0], [299, 150, 0, 1], [5, 6, 7, 8], [299, 150, 0, 1]
    t = np.tile([1.0, 0.5, -inf, 0.0], (7, 1))
    t[3] = t[6] = [3.0, -inf, -inf, -inf]
    loss, _, status = check_distill(x, ids, t, 1.0)
    assert loss[4] == inf and math.isnan(loss[3]) and status == dspark.ERR_NONFINITE
    x[3] = 0.0
    t[5] = -inf                                       # a teacher without mass: an empty list
    loss, grad, status = check_distill(x, ids, t, 1.0)
    assert loss[5] == 0 and not grad[5].any() and status == dspark.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
def test_distill_lists_masked_entries(dtype, rest, tau):
    """The teacher lists entries that the drafter's truncated row holds at the type's lowest value: their distance times
    their share, which may be past float32's range (then infinite), and the gradient of an entry without probability."""
    V, low = 600, float(torch.finfo(dtype).min)
    x = torch.full((4, V), low, dtype=dtype, device=DEV)
    x[:, 5:9] = torch.tensor([1.0, 2.0, -1.0, 0.5], dtype=dtype, device=DEV)
    ids = np.array([[5, 6, 100], [100, 101, 102], [5, 100, 101], [5, 6, 7]])
    t = np.array([[1.0, 2.0, 0.0], [3.0, 3.0, 3.0], [0.0, -9.0, 2.0], [1.0, 1.0, 1.0]])
    lse = np.log(np.exp(t / tau).sum(1) + 0.7)
    loss, grad, status = run_distill(x, ids, t, tau, lse if rest else None)
    assert status == dspark.OK
    for r in range(4):
        L, G, _ = O.distill(host(x)[r], ids[r], np.float32(t[r]), tau, np.float32(lse[r]) if rest else None)
        # the shares are within 2^-24 of the sum's terms, the logarithms within 2^-22. The largest float32 is 2^128 (1 - 2^-24),
        # infinity what rounds past it: within 2^-20 of 2^128 a value may come out as either
        if L > 2.0 ** 128 * (1 + 2.0 ** -20):
            assert loss[r] == math.inf
        else:
            near = L > 2.0 ** 128 * (1 - 2.0 ** -20) and loss[r] == math.inf
            assert near or abs(loss[r] - L) <= 2.0 ** -21 * (1 + abs(L)), (r, loss[r], L)
        assert np.abs(grad[r] - G).max() <= (HALF_STEP[dtype] + 2.0 ** -19) * (np.abs(G).max() + 2.0 ** -3)


@pytest.mark.parametrize("tau", [0.5, 2.0])
def test_distill_masked_teachers(tau):
    """Teachers' lists that hold the type's lowest value: no share beside an ordinary entry, equal shares among themselves."""
    x, ids, t, lse, _ = problem(2, 3, 200, 4, torch.float32, tau)
    low = float(np.finfo(np.float32).min)
    t[0, 1:], t[1], t[2, 3] = low, low, low
    assert check_distill(x, ids, t, tau)[2] == dspark.OK
    t[1, 0] = 1.0
    lse = np.log(np.exp(t / tau).sum(1) + 0.5)
    assert check_distill(x, ids, t, tau, lse)[2] == dspark.OK
    lse[2] = -3e38
    loss, grad, status = run_distill(x, ids, t, tau, lse)
    assert status == dspark.ERR_NONFINITE and math.isnan(loss[2]) and not grad[2].any() and np.isfinite(loss[:2]).all()


def test_distill_bad_rows():
    x, ids, t, lse, _ = problem(3, 6, 500, 4, torch.float32, 1.0)
    good = run_distill(x, ids, t, 1.0, lse)
    for change in ("x nan", "x inf", "x empty", "t nan", "t inf", "lse nan", "lse inf"):
        xb, tb, lb = x.clone(), t.copy(), lse.copy()
        what, value = change.split()
        value = {"nan": math.nan, "inf": math.inf, "empty": -math.inf}[value]
        if change == "x empty":
            xb[2] = value
        elif what == "x":
            xb[2, 77] = value
        elif what == "t":
            tb[2, 1] = value
        else:
            lb[2] = value
        loss, grad, status = run_distill(xb, ids, tb, 1.0, lb)
        assert status == dspark.ERR_NONFINITE and math.isnan(loss[2]) and not grad[2].any()
        others = [0, 1, 3, 4, 5]
        assert np.array_equal(loss[others], good[0][others]) and np.array_equal(grad[others], good[1][others])


def test_distill_unaligned():
    V = 1003
    x, ids, t, lse, _ = problem(6, 5, V, 9, torch.bfloat16, 1.0)
    want = run_distill(x, ids, t, 1.0, lse)
    for a, b in [(1, 0), (0, 3), (5, 5)]:
        y = torch.cat([x.new_zeros(a), x.flatten()])[a:].view_as(x)
        whole = torch.full((5 * V + 16,), -7.0, dtype=x.dtype, device=DEV)
        grad = whole[b:b + 5 * V].view(5, V)
        loss, ws = torch.empty(5, device=DEV), ws_small()
        dspark.distill(y, i32(ids), on(t, torch.float32), 1.0, loss, ws, grad=grad, teacher_lse=on(lse, torch.float32))
        check_distill(y, ids, t, 1.0, lse)
        assert (whole[:b] == -7).all() and (whole[b + 5 * V:] == -7).all()
        # another split over threads: sums in another order, so within both bounds
        assert np.abs(host(loss) - want[0]).max() <= 2 * (weight_error(0.0, 40.0) * 2 + 2.0 ** -20)


def test_distill_gradient_against_differences():
    """Central differences of the float32 loss along directions: the loss is within its bound (about 1e-5 here) at either
    end, so the quotient is within that over the step, and the third derivative of 8 over the step's square."""
    x, ids, t, lse, rng = problem(9, 4, 700, 12, torch.float32, 1.0)
    _, grad, _ = run_distill(x, ids, t, 1.0, lse)
    for _ in range(4):
        d = rng.normal(size=(4, 700))
        d /= np.abs(d).max()
        e = 2.0 ** -6
        up, down = (run_distill(on(host(x) + sign * e * d, torch.float32), ids, t, 1.0, lse, back=False)[0] for sign in (1, -1))
        assert np.abs((up - down) / (2 * e) - (grad * d).sum(1)).max() <= 1e-5 / e + 8 * e ** 2
