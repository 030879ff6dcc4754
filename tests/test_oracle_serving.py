"""Pins of the serving operators' oracle: worked values and properties (no GPU)."""
import math

import numpy as np

from oracle import serving as S


def test_plan_worked_example():
    # page 4; request 0: 3 cached + 6 new = 9 tokens, 3 pages, 1 held; request 1: 8 + 0; request 2: 0 + 1
    table = [[5, 0, 0], [6, 7, 0], [0, 0, 0]]
    p = S.page_plan([3, 8, 0], [6, 0, 1], [9, 2, 4, 1], 4, table, 8)
    assert p["table"].tolist() == [[5, 9, 2], [6, 7, 0], [4, 0, 0]]
    assert p["q_start"] == [0, 6, 6, 7] and p["kv_len"] == [9, 8, 1] and p["used"] == 3 and not p["short"]
    assert p["positions"] == [3, 4, 5, 6, 7, 8, 0, -1]
    assert p["slots"] == [23, 36, 37, 38, 39, 8, 16, -1]


def test_plan_short_list():
    p = S.page_plan([0, 0], [4, 4], [3], 4, [[0], [0]], 8)
    assert p["short"] and p["used"] == 1 and p["table"].tolist() == [[3], [-1]]
    assert p["slots"] == [12, 13, 14, 15, -1, -1, -1, -1]


def test_attention_equals_one_softmax():
    rng = np.random.default_rng(0)
    k, v = rng.normal(size=(6, 4, 1, 8)), rng.normal(size=(6, 4, 1, 8))
    q = rng.normal(size=(3, 2, 8))
    out, lse, _, _ = S.attention(q, k, v, np.array([5, 2]), 6, np.array([[1, 3], [4, 0]]), [0, 2, 3], [5, 1], 0.3)
    keys = np.concatenate([k[5, :, 0], k[2, :2, 0], k[1, :, 0]])  # token 0 of request 0: 6 + 4 keys
    vals = np.concatenate([v[5, :, 0], v[2, :2, 0], v[1, :, 0]])
    e = np.exp(keys @ q[0, 1] * 0.3)
    assert np.allclose(out[0, 1], e @ vals / e.sum()) and np.isclose(lse[0, 1], math.log(e.sum()))


def test_attention_empty_row():
    k = np.zeros((1, 4, 1, 8))
    out, lse, _, _ = S.attention(np.ones((2, 1, 8)), k, k, np.array([], dtype=int), 0, np.array([[0]]), [0, 2], [1], 1.0)
    assert np.isneginf(lse[0, 0]) and not out[0].any() and lse[1, 0] == 0.0


def test_rule_worked_example():
    x = [1.0, 3.0, 3.0, 0.0, -math.inf, 2.0]  # weights 1/4, 1, 1, 1/8, 0, 1/2 at rate 1
    T = math.log2(math.e)
    for k, p, mp, want in [(0, 1.0, 0.0, [0, 1, 2, 3, 5]), (1, 1.0, 0.0, [1]), (3, 1.0, 0.0, [1, 2, 5]),
                           (0, 0.3, 0.0, [1]), (0, 0.5, 0.0, [1, 2]), (3, 0.85, 0.0, [1, 2, 5]), (0, 1.0, 0.25, [0, 1, 2, 5]),
                           (0, 0.0, 0.0, [1]), (0, 1.0, 7.0, [1, 2])]:
        kept, w, _ = S.rule(x, T, k, p, mp)
        assert np.flatnonzero(kept).tolist() == want, (k, p, mp)
        assert S.exact_rule(x, 1.0, k, p, mp)[0] == want
    kept, w, _ = S.rule(x, T, 3, 1.0, 0.0)
    for u, token in [(0.0, 1), (0.39, 1), (0.41, 2), (0.81, 5), (0.999, 5)]:
        assert S.draw(kept, w, u)[0] == token
        assert S.exact_rule(x, 1.0, 3, 1.0, 0.0, u)[1] == token


def test_greedy_keeps_the_first_maximum():
    kept, _, _ = S.rule([0.0, 2.0, 2.0], 0.0, 2, 0.5, 0.0)
    assert np.flatnonzero(kept).tolist() == [1]
