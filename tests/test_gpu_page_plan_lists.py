"""dspark_page_plan with a list of free pages that ends at a negative id: nothing behind it is given out, `used` is what was taken."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import serving as S

pytestmark = pytest.mark.gpu

from test_gpu_serving import check_plan, run_plan  # noqa: E402

if torch.cuda.is_available():
    from speculative_decoding_draft_seq_gb300 import dspark


@pytest.mark.parametrize("free,taken", [([7, -1, -1], [7, -1, -1]), ([7, -1, 5], [7, -1, -1]), ([-1, 7, 5], [-1, -1, -1]),
                                        ([7, 5, 6, -1], [7, 5, 6]), ([7, 5, -3, 6], [7, 5, -1]), ([], [-1, -1, -1])])
def test_plan_takes_pages_up_to_a_negative_id(free, taken):
    table, _, _, _, slots, used, status = run_plan([4, 4, 0], [1, 2, 1], free, 4, [[1, 9], [2, 9], [9, 9]], 8)
    assert table.tolist() == [[1, taken[0]], [2, taken[1]], [taken[2], 9]]
    at = lambda x, off: -1 if x < 0 else 4 * x + off  # noqa: E731
    assert slots.tolist() == [at(taken[0], 0), at(taken[1], 0), at(taken[1], 1), at(taken[2], 0), -1, -1, -1, -1]
    assert used.item() == sum(x >= 0 for x in taken) and status == (dspark.OK if min(taken) >= 0 else dspark.ERR_CAPACITY)


@pytest.mark.parametrize("R,new,page", [(1, 900, 1), (5, 4000, 3), (128, 17, 4), (129, 40, 16), (700, 33, 8), (2049, 3, 1)])
def test_plan_with_a_list_that_ends_anywhere(R, new, page):
    """Lists that end in the first or a later CTA's requests, before and after the first 512 entries."""
    rng = np.random.default_rng(R + page)
    c, n = rng.integers(0, 50, R), rng.integers(0, new + 1, R)
    width = -(-(50 + new) // page)
    need = int(sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(c, n)))
    table = np.full((R, width), 3, dtype=np.int32)
    for capacity in (int(n.sum()), int(n.sum()) // 2):
        for end in sorted({0, 1, need // 3, min(need, 511), min(need, 512), max(need - 1, 0), need}):
            free = rng.permutation(need + 5)
            free[end] = -1  # (the ids after it stay)
            want = S.page_plan(c, n, free, page, table, capacity)
            assert want["used"] <= end
            check_plan(run_plan(c, n, free, page, table, capacity), want)


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_plan_with_a_list_at_any_alignment(offset):
    """Lists that begin at each of the four words of 16 bytes, of 0 to 9 entries, a negative id at each place."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(512, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:256]
    for n in range(10):
        for end in range(n + 1):
            ids = np.arange(100, 100 + n)
            ids[end:end + 1] = -1
            whole = i32([5] * offset + ids.tolist() + [6] * 4)
            got = [torch.full(s, -7, dtype=d, device="cuda") for s, d in [((2, 9), torch.int32), ((3,), torch.int32), ((2,), torch.int32),
                                                                          ((24,), torch.int32), ((24,), torch.int64), ((1,), torch.int32)]]
            ws.zero_()
            dspark.page_plan(i32([0, 1]), i32([9, 8]), whole[offset:offset + n], 2, *got, ws)
            check_plan((*got, dspark.device_status(ws)), S.page_plan([0, 1], [9, 8], ids, 2, np.full((2, 9), -7), 24))
