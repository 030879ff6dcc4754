"""The rounds of examples/lookup_rounds.py, followed on the host by the reference of test_gpu_serving_rounds: every emitted
token of every sample is one that the sampling rule allows after the tokens before it; no page is lost or held by
something else; the taught drafter's gradient is the divergence's."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import lookup_rounds as L  # noqa: E402
from oracle import target_pass as O  # noqa: E402
from test_gpu_serving_rounds import reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rule,kept", [((0.0, 0, 1.0, 0.0), 1), ((1.0, 5, 1.0, 0.0), 5),
                                       (([0.0, 0.7, 1.3] * 3, [2] * 9, [1.0] * 9, [0.0] * 9), 2)])
@pytest.mark.parametrize("prefix_len,page", [(100, 16), (0, 64), (64, 32)])
def test_samples_are_allowed(rule, kept, prefix_len, page):
    m = L.Model()
    rng = np.random.default_rng(prefix_len + page)
    prefix = [int(t) for t in rng.integers(0, m.V, prefix_len)]
    prompts = [[int(t) for t in rng.integers(0, 30, n)] for n in (40, 16, 33)]
    s = L.Samples(m, prefix, prompts, samples=3, rule=rule, page=page)
    for i in range(9):
        s.round()
        if i == 4:
            s.compact()
    s.check()
    for r, got in enumerate(s.emitted()):
        prompt = prompts[r // 3]
        assert len(got) >= 10 and all(0 <= x < m.V for x in got)
        first = prefix_len + len(prompt) - 1
        logits, bound = reference(m, prefix + prompt + got[:-1], first)
        for i, token in enumerate(got):
            least = np.sort(logits[i] - bound[i])[-kept]
            assert logits[i, token] + bound[i, token] >= least, (r, i)
    # a page is held by rows of one prompt, or by the prefix; the free ones are the rest
    table, cached, pinned = s.table.tolist(), s.cached.tolist(), s.pinned.tolist()
    owner = {x: "prefix" for x in pinned}
    for r in range(s.R):
        for x in table[r][:-(-cached[r] // page)]:
            assert owner.setdefault(x, r // 3) == r // 3
    s.collect(s.table, s.cached)
    refs, free, n = O.page_collect(table, cached, page, s.n_pages, pinned)
    assert s.refs.tolist() == refs and s.free.tolist() == free and n == s.n_pages - len(owner)


def test_greedy_samples_of_a_prompt_agree():
    m = L.Model()
    s = L.Samples(m, [], [[1, 2, 3, 4] * 6], samples=4, rule=(0.0, 0, 1.0, 0.0))
    for _ in range(10):
        s.round()
    s.check()
    shortest = min(map(len, s.emitted()))
    assert len({tuple(x[:shortest]) for x in s.emitted()}) == 1


@pytest.mark.parametrize("temperature", [1.0, 2.0])
def test_taught_gradient(temperature):
    g = torch.Generator().manual_seed(3)
    V, d, N = 300, 16, 40
    W, LM = torch.randn((V, d), generator=g), torch.randn((d, V), generator=g)
    previous, target = torch.randint(0, 50, (N,), generator=g), 2 * torch.randn((N, V), generator=g)
    loss, dW = L.teach(W.cuda(), LM.cuda(), previous.cuda(), target.cuda(), temperature, top=20)
    x = W.double()[previous] @ LM.double()
    want, total = torch.zeros(V, d, dtype=torch.float64), 0.0
    size = torch.zeros(V, d, dtype=torch.float64)
    for r in range(N):
        t, ids = torch.topk(target[r].double(), 20)
        lse = float(torch.logsumexp(target[r].double() / temperature, 0))
        value, grad, _ = O.distill(x[r].numpy(), ids.numpy(), t.numpy(), temperature, lse)
        total += value / N
        want[previous[r]] += LM.double() @ torch.from_numpy(grad) / N
        size[previous[r]] += LM.double().abs() @ torch.from_numpy(np.abs(grad) + 1.0 / V) / N
    # float32 throughout: the logits (d products), a weight's error of 2^-20, sums of V products: below 2^-16 of the terms
    assert (dW.cpu().double() - want).abs().max() <= 2.0 ** -16 * size.max()
    assert abs(float(loss) - total) <= 2.0 ** -16 * (1 + total)


def test_example_runs():
    L.main()
