"""Distillation lists that hold entries to which the drafter gives probability 0, among more entries than a warp has lanes.

Such an entry with a teacher's share makes the loss infinite wherever it stands in the list; the gradient and the other rows'
losses keep the bounds of test_gpu_target_pass.check_distill."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_gpu_target_pass import DTYPES, check_distill, problem, run_distill  # noqa: E402

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rest", [False, True])
# one CTA a row; several; rows that are read twice
@pytest.mark.parametrize("N,V,K", [(90, 1500, 100), (90, 2500, 1024), (3, 5000, 300), (2, 129280, 1024), (1, 300000, 400)])
def test_an_entry_without_probability_anywhere_in_a_list(dtype, rest, N, V, K):
    x, ids, t, lse, rng = problem(N + K, N, V, K, dtype, 1.0)
    ids, t = ids.astype(np.int64), t.copy()
    # the list in any order, so that every CTA and lane meets such entries before and after ordinary ones
    for r in range(N):
        order = rng.permutation(K)
        ids[r], t[r] = ids[r][order], t[r][order]
    # (rows of one entry: at the front, at the second half's front, at the end; of many; of none; without a share)
    places = [[0], [(K + 1) // 2], [K - 1], list(range(0, K, 3)), [], [0, 1]]
    for r in range(N):
        for j in places[r % 6]:
            x[r, int(ids[r, j])] = -math.inf
        if r % 6 == 5:
            t[r, :2] = -math.inf
    loss, grad, status = check_distill(x, ids, t, 1.0, lse if rest else None)
    assert status == dspark.OK
    for r in range(N):
        assert (loss[r] == math.inf) == (r % 6 < 4), (r, loss[r])
    assert np.isfinite(grad).all()
    alone = run_distill(x, ids, t, 1.0, lse if rest else None, back=False)
    over = run_distill(x.clone(), ids, t, 1.0, lse if rest else None, in_place=True)
    assert np.array_equal(alone[0], loss) and np.array_equal(over[0], loss) and np.array_equal(over[1], grad)


def test_an_entry_without_probability_beside_a_bad_row():
    """A row with NaN has loss NaN whatever else it lists; rows beside it keep theirs."""
    x, ids, t, lse, _ = problem(5, 4, 3000, 200, torch.float32, 1.0)
    x[0, int(ids[0, 0])] = -math.inf
    x[1, int(ids[1, 0])] = -math.inf
    x[1, 7] = math.nan
    loss, grad, status = run_distill(x, ids, t, 1.0, lse)
    assert loss[0] == math.inf and math.isnan(loss[1]) and np.isfinite(loss[2:]).all() and status == dspark.ERR_NONFINITE
    assert np.isfinite(grad).all() and not grad[1].any()
