"""Pins of the oracle's lists of free pages: a negative id ends one, `used` is what was taken (no GPU needed)."""
import pytest

from oracle import target_pass as O


@pytest.mark.parametrize("free,dst,used", [([1, -1, -1], [-1, 1, -1], 1), ([1, -1, 5], [-1, 1, -1], 1), ([-1, 1, 5], [-1, -1, -1], 0),
                                           ([1, 5, -1], [-1, 1, 5], 2), ([1, 5, 6, 7], [-1, 1, 5], 2), ([], [-1, -1, -1], 0)])
def test_fork(free, dst, used):
    """Three rows end inside page 2: the first keeps it, two need copies."""
    got = O.page_fork([[4, 2]], [6], [0, 0, 0], None, 4, 10, free)
    assert got["dst"] == dst and got["used"] == used and got["src"] == [-1] + [2 if x >= 0 else -1 for x in dst[1:]]
    assert got["new_table"] == [[4, 2]] + [[4, x] for x in dst[1:]]
