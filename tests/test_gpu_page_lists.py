"""Lists of free pages that end at a negative id: nothing behind it is given out, `used` is what was taken."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import target_pass as O

pytestmark = pytest.mark.gpu

from test_gpu_target_pass import SHAPES, run_fork, table_of  # noqa: E402

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark


@pytest.mark.parametrize("free,dst,used", [([1, -1, -1], [-1, 1, -1], 1), ([1, -1, 5], [-1, 1, -1], 1), ([-1, 1, 5], [-1, -1, -1], 0),
                                           ([1, 5, -1], [-1, 1, 5], 2), ([1, 5, 6, 7], [-1, 1, 5], 2), ([], [-1, -1, -1], 0),
                                           ([1, -7, 5, 6], [-1, 1, -1], 1)])
def test_fork_takes_pages_up_to_a_negative_id(free, dst, used):
    """Three rows end inside page 2: the first keeps it, two need copies."""
    got, status = run_fork(np.array([[4, 2]]), [6], [0, 0, 0], None, 4, 10, free, [])
    assert got["dst"] == dst and got["used"] == used
    assert got["new_table"] == [[4, 2]] + [[4, x] for x in dst[1:]] and got["tokens"] == [0] + [2 if x >= 0 else 0 for x in dst[1:]]
    assert status == (dspark.OK if used == 2 else dspark.ERR_CAPACITY)


@pytest.mark.parametrize("R,width,page,n_pages,share", SHAPES)
def test_fork_with_a_list_that_ends_anywhere(R, width, page, n_pages, share):
    rng = np.random.default_rng(R + n_pages)
    table, kv_len, spare = table_of(rng, R, width, page, n_pages, share)
    n = R + R // 3 + 1
    parent = rng.integers(-1, R, n)
    for end in sorted({0, 1, min(n // 7, len(spare)), min(n // 2, len(spare)), len(spare)}):
        free = spare.copy()
        free[end:end + 1] = -1  # (the ids after it stay)
        want = O.page_fork(table, kv_len, parent, None, page, n_pages, free, [])
        got, status = run_fork(table, kv_len, parent, None, page, n_pages, free, [])
        assert got == want and want["used"] <= end
        short = any(row[-(-m // page) - 1] < 0 for row, m in zip(want["new_table"], want["new_len"]) if m)
        assert status == (dspark.ERR_CAPACITY if short else dspark.OK)
