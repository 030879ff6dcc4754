"""Pins of the oracle of what follows the target's pass (no GPU needed)."""
import itertools
import math
from collections import Counter
from fractions import Fraction

import numpy as np
import pytest

from oracle import target_pass as O


def test_softmax_special_rows():
    inf = math.inf
    assert O.softmax([1.0, 3.0, 3.0], 0.0)[0].tolist() == [0, 1, 0]
    assert O.softmax([1.0, -inf, 5.0], inf)[0].tolist() == [0.5, 0, 0.5]
    assert O.softmax([-inf, -inf], 1.0)[0].tolist() == [0, 0] and O.softmax([math.nan, 1.0], 1.0)[0].tolist() == [0, 0]
    p, y = O.softmax([0.0, 2.0, -1.0], 0.5)
    assert np.allclose(p, np.exp([0, 4, -2]) / np.exp([0, 4, -2]).sum()) and y[1] == 0


@pytest.mark.parametrize("with_rows", [True, False])
def test_verified_block_has_the_targets_law(with_rows):
    """Two drafts over three tokens, the uniforms on an even grid fine enough to be exact: the first emitted token's law is
    the target's first row, whatever the drafter's."""
    n = 60
    P = [np.array(a, dtype=np.float32) / 64 for a in ([32, 16, 16], [8, 40, 16], [16, 16, 32])]
    Q = [np.array(a, dtype=np.float32) / 64 for a in ([16, 32, 16], [32, 8, 24])]
    grid = [(2 * i + 1) / (2 * n) for i in range(n)]
    law = Counter()
    firsts = [(v, Fraction(float(Q[0][v]))) for v in range(3)] if with_rows else [(1, Fraction(1))]
    for x0, weight in firsts:
        for u0, u2 in itertools.product(grid, grid):
            tokens = np.array([[x0, 2]])
            draft = np.stack(Q)[None] if with_rows else None
            out, acc, p_tok = O.verify_probs(np.stack(P), [0, 3], draft, tokens, np.array([[u0, 0.999, u2]]))
            law[int(out[0, 0])] += weight / n ** 2
            assert p_tok[0].tolist() == [P[0][x0], P[1][2]]
            assert acc[0] <= 2 and (out[0, acc[0] + 1:] == -1).all()
    for v in range(3):
        assert abs(float(law[v]) - float(P[0][v])) < 1.0 / n


def test_draw_is_the_inverse_cdf():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25], dtype=np.float32)
    assert [O.draw(w, u) for u in (0.0, 0.249, 0.25, 0.74, 0.75, 1 - 2.0 ** -53)] == [1, 1, 3, 3, 4, 4]
    assert O.draw(w * 0, 0.5) == -1 and O.draw(np.array([math.nan, -1.0, 2.0]), 0.9) == 2


def test_verify_without_mass_and_bad_rows():
    P = np.array([[0.5, 0.5], [0.0, 0.0]], dtype=np.float32)
    # the draft's row equals the target's: the residual has no mass, the draw is from the target
    out, acc, _ = O.verify_probs(P, [0, 2], np.array([[[0.5, 0.5]]], dtype=np.float32), np.array([[0]]), np.array([[0.999999, 0.7]]))
    assert acc[0] == 1 and out[0].tolist() == [0, -1]
    out, acc, _ = O.verify_probs(P[:1], [0, 2], None, np.array([[0]]), np.array([[0.1, 0.1]]))
    assert acc[0] == 0 and out[0].tolist() == [-1, -1]


def _random_rows(rng, R, width, page, n_pages, shared):
    ids = rng.permutation(n_pages)
    kv_len = rng.integers(0, width * page + 1, R)
    table, at = np.full((R, width), -1), 0
    for r in range(R):
        n = -(-kv_len[r] // page)
        s = min(n, shared, kv_len[0] // page) if r else 0
        table[r, :s] = table[0, :s]
        table[r, s:n] = ids[at:at + n - s]
        at += n - s
    return table, kv_len, ids[at:]


@pytest.mark.parametrize("seed", range(6))
def test_page_calls_keep_what_rows_read(seed):
    """Tokens are written into a cache through the table; forked and compacted rows read the same tokens through theirs,
    a written token shows in one row only, and free pages are nobody's."""
    rng = np.random.default_rng(seed)
    page, width, R, n_pages = 4, 5, 6, 60
    table, kv_len, spare = _random_rows(rng, R, width, page, n_pages, 2)
    pinned = [int(spare[0])]
    cache = rng.integers(1, 1 << 30, (n_pages, page))
    read = lambda row, n: [int(cache[row[i // page], i % page]) for i in range(n)]  # noqa: E731
    refs, free, n_free = O.page_collect(table, kv_len, page, n_pages, pinned)
    assert n_free == sum(x >= 0 for x in free) and all(refs[x] == 0 for x in free[:n_free]) and refs[pinned[0]] == 1
    parent = rng.integers(-1, R, 9)
    length = [0 if q < 0 else int(rng.integers(0, kv_len[q] + 1)) for q in parent]
    f = O.page_fork(table, kv_len, parent, length, page, n_pages, free[:n_free], pinned)
    want = [read(table[q], n) for q, n in zip(parent, length)]
    for a, b, n in zip(f["src"], f["dst"], f["tokens"]):
        if a >= 0:
            assert refs[b] == 0
            cache[b, :n] = cache[a, :n]
    assert [read(row, n) for row, n in zip(f["new_table"], f["new_len"])] == want
    # one more token into every row that ends inside a page: no other row sees it
    for i, (row, n) in enumerate(zip(f["new_table"], f["new_len"])):
        if n % page:
            cache[row[n // page], n % page] = -i - 1
            want[i].append(-i - 1)
    lens = [len(w) for w in want]
    assert [read(row, n) for row, n in zip(f["new_table"], lens)] == want
    c = O.page_compact(f["new_table"], lens, page, n_pages, pinned)
    for a, b in zip(c["src"], c["dst"]):
        if a >= 0:
            cache[b] = cache[a]
    assert [read(row, n) for row, n in zip(c["new_table"], lens)] == want
    assert max([x for row in c["new_table"] for x in row] + c["new_pinned"]) < c["n_live"]
    refs, _, n_free = O.page_collect(c["new_table"], lens, page, n_pages, c["new_pinned"])
    assert n_free == n_pages - c["n_live"] and all(refs[:c["n_live"]])


@pytest.mark.parametrize("seed,rest", [(s, r) for s in range(4) for r in (False, True)])
def test_distill_gradient_is_the_losss_difference(seed, rest):
    rng = np.random.default_rng(seed)
    V, K, tau = 23, 6, (0.7, 1.0, 2.5, 1.5)[seed]
    x, full = rng.normal(size=V) * 2, rng.normal(size=V) * 2
    ids = rng.permutation(V)[:K]
    ids[K - 1] = [-1, ids[0], ids[K - 1], -1][seed]  # a padded list, an id that comes twice
    t = full[ids]
    lse = math.log(np.exp(full / tau).sum()) if rest else None
    loss, grad, parts = O.distill(x, ids, t, tau, lse)
    e = 1e-6
    for v in range(V):
        step = np.eye(V)[v] * e
        d = (O.distill(x + step, ids, t, tau, lse)[0] - O.distill(x - step, ids, t, tau, lse)[0]) / (2 * e)
        # central differences: e^2 / 6 times a third derivative below 8 / tau^3, and 2^-52 |loss| / e of rounding
        assert abs(d - grad[v]) < 2 * e ** 2 / tau ** 3 + 2.0 ** -50 * (1 + abs(loss)) / e
    assert abs(grad.sum()) < 1e-12 and loss > -1e-12 or seed == 1
    if not rest:
        assert abs(parts["p"].sum() - 1) < 1e-12


def test_distill_special_rows():
    x = np.array([0.0, 1.0, 2.0])
    assert O.distill(x, [-1, -1], [5.0, 5.0], 1.0)[0] == 0 and not O.distill(x, [-1], [5.0], 1.0)[1].any()
    loss, grad, _ = O.distill(x, [-1], [5.0], 1.0, lse=0.0)
    assert abs(loss) < 1e-15 and np.abs(grad).max() < 1e-15
    loss, grad, _ = O.distill(x, [0, 1, 2], x, 2.0)  # the teacher is the drafter
    assert abs(loss) < 1e-15 and np.abs(grad).max() < 1e-15
    assert O.distill([0.0, -math.inf], [1], [0.0], 1.0)[0] == math.inf
