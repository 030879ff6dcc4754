"""The rounds of examples/serving_rounds.py, followed on the host: every emitted token has to be one that the
target's sampling rule allows after the tokens before it, by a plain forward pass in float64.

The device rounds to bf16 at q, k, v, the attention's weights and output, its product with Wo, the hidden
state and the logits: independent relative errors of at most 2^-9 each. A logit's error is a sum of many of
them, taken as six times the root of the sum of their squares: two roundings of each hidden element (the
product with Wo and the sum), four of each attention output's share in it (v, weight, scores, output), and
the logit's own rounding, at most 2^-8 of it with the comparison's other side.
"""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import serving_rounds as S  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -9


def reference(m, tokens, first):
    """(logits, error bounds) of the token after each position from `first` on, in float64."""
    f = {k: getattr(m, k).double().cpu().numpy() for k in ("E", "P", "Wq", "Wk", "Wv", "Wo", "LM")}
    t = np.array(tokens)
    x = f["E"][t] + f["P"][np.arange(len(t))]
    q = (x[first:] @ f["Wq"]).reshape(-1, m.Hq, m.D)
    k, v = ((x @ f[n]).reshape(-1, m.Hkv, m.D).repeat(m.Hq // m.Hkv, axis=1) for n in ("Wk", "Wv"))
    s = np.einsum("thd,nhd->thn", q, k) * m.D ** -0.5
    s[np.broadcast_to((np.arange(len(t))[None] > np.arange(first, len(t))[:, None])[:, None], s.shape)] = -np.inf
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    out = np.einsum("thn,nhd->thd", w, v).reshape(len(t) - first, -1)
    share = np.sqrt(np.einsum("thn,nhd->thd", w ** 2, v ** 2)).reshape(len(t) - first, -1)
    h = f["E"][t[first:]] + out @ f["Wo"]
    dh2 = (2 * EPS * h) ** 2 + (4 * EPS) ** 2 * (np.maximum(np.abs(out), share) ** 2 @ f["Wo"] ** 2)
    logits = h @ f["LM"]
    return logits, 6 * np.sqrt(dh2 @ f["LM"] ** 2) + 2 * EPS * np.abs(logits)


@pytest.mark.parametrize("rule,kept", [((0.0, 0, 1.0, 0.0), 1), ((1.0, 5, 1.0, 0.0), 5), ((0.7, 3, 0.9, 0.05), 3)])
@pytest.mark.parametrize("prefix_len,page", [(200, 16), (0, 64), (64, 32)])
def test_emitted_tokens_are_allowed(rule, kept, prefix_len, page):
    m = S.Model()
    rng = np.random.default_rng(prefix_len + page)
    prefix = [int(t) for t in rng.integers(0, m.V, prefix_len)]
    prompts = [[int(t) for t in rng.integers(0, m.V, n)] for n in (1, 2, 17, 40, 64, 33, 9)]
    server = S.Server(m, prefix, prompts, rule=rule, page=page)
    accepted = np.array([server.round() for _ in range(8)])
    assert accepted.sum() > 0 and (accepted < server.gamma).any()

    for r, prompt in enumerate(prompts):
        got = server.emitted[r]
        assert len(got) == 1 + (accepted[:, r] + 1).sum() and all(0 <= x < m.V for x in got)
        first = prefix_len + len(prompt) - 1
        logits, bound = reference(m, prefix + prompt + got[:-1], first)
        for i, token in enumerate(got):
            least = np.sort(logits[i] - bound[i])[-kept]  # at least `kept` entries reach this
            assert logits[i, token] + bound[i, token] >= least, (r, i)

    # no page is lost and none is held twice
    table, cached = server.table.cpu().numpy(), server.cached.cpu().numpy()
    held = [int(x) for r in range(len(prompts)) for x in table[r, :-(-cached[r] // page)]]
    held += [int(x) for x in server.prefix_pages.cpu().numpy().ravel()]
    assert sorted(held + [int(x) for x in server.free]) == list(range(server.k_cache.shape[0]))


def test_rounds_repeat_bit_for_bit():
    m = S.Model()
    prompts = [[5, 6, 7], list(range(30))]
    runs = []
    for _ in range(2):
        server = S.Server(m, list(range(100, 180)), prompts)
        for _ in range(5):
            server.round()
        runs.append(server.emitted)
    assert runs[0] == runs[1]
