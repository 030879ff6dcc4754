"""The calls after the target's pass as a serving engine uses them: one after the other on one stream, captured in a
graph and replayed on other inputs, on a stream of their own, on caches past 2^32 elements, with rows behind the last one
left as they were, repeated bit for bit."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import target_pass as O

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark

from test_gpu_target_pass import DEV, blank, block, check_distill, host, i32, on, problem, run_distill, table_of, ws_small


def verify_buffers(R, gamma):
    return blank(R, gamma + 1), blank(R), blank(R, gamma, dtype=torch.float32)


def test_round_after_the_targets_pass():
    """Logits of several temperatures -> truncated rows -> probabilities -> verification -> the lengths that stay -> free
    pages -> forks with their copies -> the front of the cache, all on the device; every step against the oracle."""
    rng = np.random.default_rng(11)
    R, gamma, V, page, width, n_pages = 6, 4, 900, 16, 6, 60
    n = np.array([5, 3, 1, 4, 5, 2])
    T, q_start = int(n.sum()), np.concatenate([[0], np.cumsum(n)])
    ws, wsp = ws_small(), dspark.new_page_workspace(n_pages)
    temps = rng.choice([0.0, 0.7, 1.0, 1.4], R)
    logits = on(rng.normal(size=(T, V)) * 3, torch.bfloat16)
    q_logits = on(rng.normal(size=(R * gamma, V)) * 3, torch.bfloat16)
    f32 = lambda a: on(np.asarray(a, dtype=np.float32), torch.float32)  # noqa: E731
    rule = [f32(np.repeat(temps, n)), i32([50] * T), f32([0.9] * T), f32([0.0] * T)]
    cut = torch.empty_like(logits)
    dspark.truncate(logits, *rule, cut, ws)
    P, Q = torch.empty((T, V), device=DEV), torch.empty((R * gamma, V), device=DEV)
    dspark.probabilities(cut, rule[0], P, ws)
    dspark.probabilities(q_logits, f32(np.repeat(temps, gamma)), Q, ws)
    assert bool(((P.cpu() > 0) <= (cut.float().cpu() > -1e38)).all())  # what the rule masked has no probability
    Q = Q.view(R, gamma, V)
    tokens = np.array([[int(Q[r, k].argmax()) if rng.random() < 0.5 else int(rng.choice(V, p=host(Q[r, k]) / host(Q[r, k]).sum()))
                        for k in range(gamma)] for r in range(R)])
    u = rng.random((R, gamma + 1))
    out, acc, p_tok = verify_buffers(R, gamma)
    dspark.verify_probs(P, i32(q_start), Q, i32(tokens), on(u, torch.float64), out, acc, p_tok, ws)
    want = O.verify_probs(P.cpu().numpy(), q_start, Q.cpu().numpy(), tokens, u)
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(acc.cpu().numpy(), want[1])

    # the cache: each request held `cached` tokens, its round's n were appended, the accepted ones and the anchor stay
    cached = rng.integers(1, width * page - gamma - 1, R)
    ids, at = rng.permutation(n_pages), 0
    table = np.full((R, width), -1)
    for r in range(R):
        need = -(-(cached[r] + n[r]) // page)
        table[r, :need], at = ids[at:at + need], at + need
    k = on(rng.normal(size=(2, n_pages, page, 2, 8)), torch.bfloat16)
    v = on(rng.normal(size=(2, n_pages, page, 2, 8)), torch.bfloat16)
    keep = i32(cached) + acc + 1
    kept = keep.tolist()
    before = [[k[:, table[r, i // page], i % page].clone() for i in range(kept[r])] for r in range(R)]
    d_table, refs, free, n_free = i32(table), blank(n_pages), blank(n_pages), blank(1)
    dspark.page_collect(d_table, keep, page, refs, free, n_free, wsp)
    assert refs.tolist() == O.page_collect(table, kept, page, n_pages)[0]

    # two samples of requests 0 and 3, request 1 dropped; the free list goes in as it came out, -1 at its end
    parent = [0, 0, 2, 3, 3, 4, 5]
    new, new_len = blank(len(parent), width), blank(len(parent))
    src, dst, count, used = blank(len(parent)), blank(len(parent)), blank(len(parent)), blank(1)
    dspark.page_fork(d_table, keep, i32(parent), None, page, n_pages, free, new, new_len, src, dst, count, used, wsp)
    dspark.page_copy(src, dst, k, v, wsp, tokens=count)
    assert used.item() == sum(kept[p] % page != 0 for p in (0, 3))
    moves, to, n_live = blank(n_pages // 2), blank(n_pages // 2), blank(1)
    dspark.page_compact(new, new_len, page, n_pages, new, moves, to, n_live, wsp)
    dspark.page_copy(moves, to, k, v, wsp)
    assert dspark.device_status(ws) == dspark.OK and dspark.device_status(wsp) == dspark.OK
    rows = new.tolist()
    for row, p in zip(rows, parent):
        assert all(torch.equal(k[:, row[i // page], i % page], before[p][i]) for i in range(kept[p]))
    assert max(x for row in rows for x in row) < n_live.item()

    # the next round's pages come from the same list
    dspark.page_collect(new, new_len, page, refs, free, n_free, wsp)
    m = len(parent)
    plan = [blank(m + 1), blank(m), blank(m * 3), blank(m * 3, dtype=torch.int64), blank(1)]
    grow = torch.full((m,), 3, dtype=torch.int32, device=DEV)
    dspark.page_plan(new_len, grow, free, page, new, *plan, ws)
    slots = plan[3].tolist()
    assert len(set(slots)) == 3 * m and min(slots) >= 0 and dspark.device_status(ws) == dspark.OK


def test_page_plan_takes_a_list_that_ends_early():
    free, ws = i32([7, -1, -1]), ws_small()
    table = i32([[1, -1], [2, -1]])
    got = [blank(3), blank(2), blank(8), blank(8, dtype=torch.int64), blank(1)]
    dspark.page_plan(i32([4, 4]), i32([1, 1]), free, 4, table, *got, ws)
    assert dspark.device_status(ws) == dspark.ERR_CAPACITY and table.tolist() == [[1, 7], [2, -1]]
    assert got[3].tolist()[:2] == [28, -1]


def test_captured_and_replayed():
    """A graph of the calls on other inputs, and on the same inputs twice: the eager calls' bits."""
    R, gamma, V = 9, 3, 4099
    blocks = [block(s, R, gamma, V, torch.float32) for s in (1, 2)]
    T = max(b[0].shape[0] for b in blocks)
    x, ids, t, lse, _ = problem(5, 12, V, 7, torch.bfloat16, 1.0)
    rng = np.random.default_rng(1)
    page, n_pages = 16, 400
    tables = [table_of(rng, 20, 9, page, n_pages, 2) for _ in range(2)]
    s = {"target": torch.zeros((T, V), device=DEV), "q_start": i32([0] * (R + 1)), "draft": torch.zeros((R, gamma, V), device=DEV),
         "tokens": i32([[0] * gamma] * R), "u": torch.zeros((R, gamma + 1), dtype=torch.float64, device=DEV), "logits": torch.zeros_like(x),
         "table": i32(tables[0][0] * 0), "kv_len": i32([0] * 20)}
    out, ws, wsp = verify_buffers(R, gamma), ws_small(), dspark.new_page_workspace(n_pages)
    probs, loss, grad = torch.empty((12, V), device=DEV), torch.empty(12, device=DEV), torch.empty_like(x)
    refs, free, n_free = blank(n_pages), blank(n_pages), blank(1)
    new, new_len, pair, count, used = blank(20, 9), blank(20), [blank(20), blank(20)], blank(20), blank(1)
    moves, n_live = [blank(n_pages // 2), blank(n_pages // 2)], blank(1)
    d_ids, d_t, d_T = i32(ids), on(t, torch.float32), torch.full((12,), 0.8, device=DEV)
    parent = i32(rng.integers(0, 20, 20))

    def step():
        dspark.verify_probs(s["target"], s["q_start"], s["draft"], s["tokens"], s["u"], *out, ws)
        dspark.probabilities(s["logits"], d_T, probs, ws)
        dspark.distill(s["logits"], d_ids, d_t, 1.0, loss, ws, grad=grad)
        dspark.page_collect(s["table"], s["kv_len"], page, refs, free, n_free, wsp)
        dspark.page_fork(s["table"], s["kv_len"], parent, None, page, n_pages, free, new, new_len, *pair, count, used, wsp)
        dspark.page_compact(new, new_len, page, n_pages, new, *moves, n_live, wsp)
        return [a.clone() for a in (*out, probs, loss, grad, refs, free, n_free, new, new_len, *pair, count, used, *moves, n_live)]

    def load(i):
        b = blocks[i]
        s["target"][:b[0].shape[0]] = b[0]
        s["q_start"].copy_(i32(b[1]))
        s["draft"].copy_(b[2])
        s["tokens"].copy_(i32(b[3]))
        s["u"].copy_(on(b[4], torch.float64))
        s["logits"].copy_(x if i == 0 else x.flip(0))
        s["table"].copy_(i32(tables[i][0]))
        s["kv_len"].copy_(i32(tables[i][1]))

    want = []
    for i in (0, 1):
        load(i)
        want.append(step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for i in (1, 0, 0):
        load(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    assert dspark.device_status(ws) == dspark.OK and dspark.device_status(wsp) == dspark.OK


def test_first_call_of_its_kind_captured():
    """Nothing a call looks up or sets on its first use is forbidden in a capture."""
    x, ids, t, _, _ = problem(6, 5, 70001, 13, torch.float32, 1.0)
    loss, grad, ws = torch.zeros(5, device=DEV), torch.zeros_like(x), ws_small()
    d_ids, d_t = i32(ids), on(t, torch.float32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        dspark.distill(x, d_ids, d_t, 1.0, loss, ws, grad=grad)
    graph.replay()
    torch.cuda.synchronize()
    want = run_distill(x, ids, t, 1.0)
    assert np.array_equal(host(loss), want[0]) and np.array_equal(host(grad), want[1])


@pytest.mark.parametrize("V", [1003, 300001])
def test_probabilities_in_place(V):
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn((4, V), generator=g, device=DEV)
    T, ws, p = on(np.array([1.0, 0.0, 0.5, math.inf], dtype=np.float32), torch.float32), ws_small(), torch.empty((4, V), device=DEV)
    dspark.probabilities(x, T, p, ws)
    dspark.probabilities(x, T, x, ws)
    assert torch.equal(x, p)


def test_page_fork_of_a_row_longer_than_its_table():
    table, got, ws = i32([[4, 2], [3, 1]]), [blank(2, 2)] + [blank(2) for _ in range(4)] + [blank(1)], dspark.new_page_workspace(10)
    dspark.page_fork(table, i32([9, 4]), i32([0, 1]), None, 4, 10, i32([0]), *got, ws)
    assert dspark.device_status(ws) == dspark.ERR_RANGE and got[0].tolist() == [[4, 2], [3, -1]] and got[1].tolist() == [8, 4]


def test_two_streams_with_a_workspace_each():
    x, ids, t, lse, _ = problem(3, 300, 2000, 16, torch.float32, 1.0)
    b = block(4, 30, 4, 2000, torch.float32)
    want_v = O.verify_probs(b[0].cpu().numpy(), b[1], b[2].cpu().numpy(), b[3], b[4])
    want_d = run_distill(x, ids, t, 1.0, lse)
    streams, ws = [torch.cuda.Stream() for _ in range(2)], [ws_small() for _ in range(2)]
    loss, grad, out = torch.empty(300, device=DEV), torch.empty_like(x), verify_buffers(30, 4)
    d = [i32(ids), on(t, torch.float32), on(lse, torch.float32), i32(b[1]), i32(b[3]), on(b[4], torch.float64)]
    torch.cuda.synchronize()
    for _ in range(20):
        dspark.distill(x, d[0], d[1], 1.0, loss, ws[0], grad=grad, teacher_lse=d[2], stream=streams[0])
        dspark.verify_probs(b[0], d[3], b[2], d[4], d[5], *out, ws[1], stream=streams[1])
    torch.cuda.synchronize()
    assert np.array_equal(host(loss), want_d[0]) and np.array_equal(host(grad), want_d[1])
    assert np.array_equal(out[0].cpu().numpy(), want_v[0])


@pytest.mark.parametrize("N,V", [(1, 50000), (37, 9001), (2500, 515)])
def test_repeats_are_the_same_bits(N, V):
    x, ids, t, lse, _ = problem(N, N, V, 33, torch.bfloat16, 0.9)
    first, T = run_distill(x, ids, t, 0.9, lse), torch.full((N,), 0.9, device=DEV)
    p0, ws = torch.empty((N, V), device=DEV), ws_small()
    dspark.probabilities(x, T, p0, ws)
    for _ in range(10):
        again, p = run_distill(x, ids, t, 0.9, lse), torch.empty((N, V), device=DEV)
        dspark.probabilities(x, T, p, ws)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1]) and torch.equal(p, p0)


def test_a_workspace_may_be_shared_by_later_calls_of_other_sizes():
    """Calls in turn on one workspace of the largest size; an earlier error stays until it is cleared."""
    rng = np.random.default_rng(8)
    ws = dspark.new_page_workspace(5000)
    for n_pages in (5000, 10, 700, 5000):
        table, kv_len, _ = table_of(rng, 5, 4, 16, n_pages)
        refs, free, n = blank(n_pages), blank(n_pages), blank(1)
        dspark.page_collect(i32(table), i32(kv_len), 16, refs, free, n, ws)
        want = O.page_collect(table, kv_len, 16, n_pages)
        assert refs.tolist() == want[0] and free.tolist() == want[1] and n.item() == want[2]
        dspark.probabilities(torch.zeros((2, 50), device=DEV), torch.ones(2, device=DEV), torch.empty((2, 50), device=DEV), ws)
    assert dspark.device_status(ws) == dspark.OK
    dspark.probabilities(torch.full((1, 50), math.nan, device=DEV), torch.ones(1, device=DEV), torch.empty((1, 50), device=DEV), ws)
    dspark.page_collect(i32(table), i32(kv_len), 16, refs, free, n, ws)
    assert dspark.device_status(ws) == dspark.ERR_NONFINITE


def test_large_page_calls_in_turn_on_one_workspace():
    """Calls over the whole GPU, whose CTAs meet at a word of the workspace: one after the other, in a graph, between calls
    of one cluster."""
    rng = np.random.default_rng(12)
    R, width, page, n_pages = 3000, 30, 16, 60000
    table, kv_len, spare = table_of(rng, R, width, page, n_pages, 3)
    parent, free = rng.integers(-1, R, R), spare
    ws, small = dspark.new_page_workspace(n_pages), table_of(rng, 4, 3, 16, 50)
    d = [i32(table), i32(kv_len), i32(parent), i32(free)]
    refs, list_, n = blank(n_pages), blank(n_pages), blank(1)
    new, new_len, pair, count, used = blank(R, width), blank(R), [blank(R), blank(R)], blank(R), blank(1)
    moved, moves, live = blank(R, width), [blank(n_pages // 2), blank(n_pages // 2)], blank(1)

    def step():
        dspark.page_collect(d[0], d[1], page, refs, list_, n, ws)
        dspark.page_fork(d[0], d[1], d[2], None, page, n_pages, d[3], new, new_len, *pair, count, used, ws)
        dspark.page_compact(d[0], d[1], page, n_pages, moved, *moves, live, ws)

    def check():
        want = O.page_collect(table, kv_len, page, n_pages)
        assert refs.tolist() == want[0] and list_.tolist() == want[1] and n.item() == want[2]
        want = O.page_fork(table, kv_len, parent, None, page, n_pages, free)
        assert new.tolist() == want["new_table"] and pair[0].tolist() == want["src"] and pair[1].tolist() == want["dst"]
        want = O.page_compact(table, kv_len, page, n_pages)
        assert moved.tolist() == want["new_table"] and moves[0].tolist() == want["src"] and live.item() == want["n_live"]
        for t in (refs, list_, n, new, *pair, moved, *moves, live):
            t.fill_(-9)

    for _ in range(3):
        step()
        check()
        small_refs, small_free = blank(50), blank(50)
        dspark.page_collect(i32(small[0]), i32(small[1]), 16, small_refs, small_free, n, ws)
        assert small_refs.tolist() == O.page_collect(small[0], small[1], 16, 50)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check()
    assert dspark.device_status(ws) == dspark.OK


def test_page_copy_past_2_32_elements():
    n_pages, page, H, D = 2 ** 17 + 3, 16, 16, 128  # 2^32 elements and more a cache
    k = torch.zeros((n_pages, page, H, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[n_pages - 1], v[5] = 3.0, 4.0
    ws = ws_small()
    dspark.page_copy(i32([n_pages - 1, 5]), i32([1, n_pages - 2]), k, v, ws)
    assert (k[1] == 3).all() and (v[n_pages - 2] == 4).all() and (k[n_pages - 2] == 0).all()
    assert int(k.count_nonzero()) == 2 * page * H * D and int(v.count_nonzero()) == 2 * page * H * D
    assert dspark.device_status(ws) == dspark.OK


def test_rows_past_2_32_bytes():
    """Row offsets past 2^31 elements in every tensor of rows."""
    N, V = 17000, 129280
    x = torch.zeros((N, V), dtype=torch.bfloat16, device=DEV)
    x[N - 1, 7], x[N - 1, V - 1] = 4.0, 5.0
    p, ws = torch.empty((N, V), dtype=torch.bfloat16, device=DEV), ws_small()
    dspark.probabilities(x, torch.ones(N, device=DEV), p, ws)
    want, _ = O.softmax(host(x[N - 1]), 1.0)
    assert np.abs(host(p[N - 1]) - want).max() <= 2.0 ** -8 * want.max() and float(p[N - 2].float().std()) == 0
    ids = torch.zeros((N, 1), dtype=torch.int32, device=DEV)
    ids[N - 1] = V - 1
    loss = torch.empty(N, device=DEV)
    dspark.distill(x, ids, torch.ones((N, 1), device=DEV), 1.0, loss, ws, grad=p)
    assert abs(float(loss[N - 1]) + math.log(want[V - 1])) < 1e-5 and abs(float(loss[0]) - math.log(V)) < 1e-5
    check_distill(x[N - 2:], ids[N - 2:].cpu().numpy(), np.ones((2, 1)), 1.0)
    g = O.distill(host(x[N - 1]), [V - 1], [1.0], 1.0)[1]
    assert np.abs(host(p[N - 1]) - g).max() <= 2.0 ** -8 * np.abs(g).max()
    u = torch.full((1, 2), 0.5, dtype=torch.float64, device=DEV)
    out = verify_buffers(1, 1)
    q = torch.zeros((1, 1, V), dtype=torch.bfloat16, device=DEV)
    q[0, 0, 3] = 1.0
    onehot = x.zero_()
    onehot[N - 2, V - 2] = 1.0
    starts = i32([N - 2, N])
    dspark.verify_probs(onehot, starts, q, i32([[3]]), u, *out, ws)
    assert out[0].tolist() == [[V - 2, -1]] and out[1].item() == 0 and dspark.device_status(ws) == dspark.OK


def test_rows_behind_the_last_are_left():
    """Rows of a round's buffers that belong to no request, and table rows that are not passed, keep their bits."""
    V = 300
    P = torch.full((10, V), 1.0 / V, device=DEV)
    P[6:] = math.nan  # past q_start[R]: never read
    out, ws = verify_buffers(2, 3), ws_small()
    dspark.verify_probs(P, i32([0, 4, 6]), None, i32([[1, 2, 3]] * 2), torch.full((2, 4), 0.25, dtype=torch.float64, device=DEV), *out, ws)
    assert dspark.device_status(ws) == dspark.OK and out[2][1].tolist()[1:] == [0.0, 0.0]
    whole = torch.full((6, V), 7.0, device=DEV)
    dspark.probabilities(whole[1:4].clone(), torch.ones(3, device=DEV), whole[1:4], ws)
    assert (whole[0] == 7).all() and (whole[4:] == 7).all()


def test_refused_views():
    x = torch.zeros((4, 20), device=DEV)
    T, ws = torch.ones(4, device=DEV), ws_small()
    with pytest.raises(ValueError, match="contiguous"):
        dspark.probabilities(x[:, ::2], T, torch.empty((4, 10), device=DEV), ws)
    with pytest.raises(TypeError):
        dspark.probabilities(x.half(), T, torch.empty((4, 20), device=DEV), ws)
    with pytest.raises(TypeError):
        dspark.probabilities(x, T.double(), torch.empty((4, 20), device=DEV), ws)
    with pytest.raises(ValueError, match="CUDA"):
        dspark.probabilities(x, T.cpu(), torch.empty((4, 20), device=DEV), ws)
    with pytest.raises(dspark.DSparkError):
        dspark.distill(x, i32([[0]] * 4), T[:, None].contiguous(), 0.0, T.clone(), ws)
    empty = torch.empty((0, 20), device=DEV)
    dspark.probabilities(empty, T[:0], empty.clone(), ws)
    dspark.distill(empty, i32(np.zeros((0, 3))), torch.empty((0, 3), device=DEV), 1.0, T[:0], ws, grad=empty.clone())
    assert dspark.device_status(ws) == dspark.OK
