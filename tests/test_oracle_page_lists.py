"""Pins of the oracle's lists of free pages: a negative id ends one, `used` is what was taken (no GPU needed)."""
import pytest

from oracle import serving as S
from oracle import target_pass as O


@pytest.mark.parametrize("free,dst,used", [([1, -1, -1], [-1, 1, -1], 1), ([1, -1, 5], [-1, 1, -1], 1), ([-1, 1, 5], [-1, -1, -1], 0),
                                           ([1, 5, -1], [-1, 1, 5], 2), ([1, 5, 6, 7], [-1, 1, 5], 2), ([], [-1, -1, -1], 0)])
def test_fork(free, dst, used):
    """Three rows end inside page 2: the first keeps it, two need copies."""
    got = O.page_fork([[4, 2]], [6], [0, 0, 0], None, 4, 10, free)
    assert got["dst"] == dst and got["used"] == used and got["src"] == [-1] + [2 if x >= 0 else -1 for x in dst[1:]]
    assert got["new_table"] == [[4, 2]] + [[4, x] for x in dst[1:]]


@pytest.mark.parametrize("free,taken", [([7, -1, -1], [7, -1]), ([7, -1, 5], [7, -1]), ([-1, 7, 5], [-1, -1]), ([7, 5, -1], [7, 5]),
                                        ([7], [7, -1]), ([], [-1, -1])])
def test_plan(free, taken):
    got = S.page_plan([4, 0], [1, 2], free, 4, [[1, 9], [9, 9]], 4)
    assert got["table"].tolist() == [[1, taken[0]], [taken[1], 9]]
    assert got["used"] == sum(x >= 0 for x in taken) and got["short"] == (min(taken) < 0)
