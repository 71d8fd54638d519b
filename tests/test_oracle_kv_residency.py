"""The oracle's cache write where tokens are not resident: their values elsewhere keep their meaning."""
import numpy as np

from oracle import kv as OK


def _cache(table, N, block, page):
    rows = np.full((8, page, 1, 16), 0x38, np.uint8)              # 1.0
    return OK.Cache(rows, np.ones((1, -(-N // block), 1)), np.array([table]), N, block, page, 0)


def test_growing_block_with_an_earlier_token_away_is_left_alone():
    c = _cache([-1, 3], 8, 8, 4)
    before = c.rows.copy()
    big = np.full((1, 2, 1, 16), 1e6)
    assert OK.write(c, big, [5], [2])
    assert c.scale[0, 0, 0] == 1.0 and np.array_equal(c.rows, before)
    small = np.full((1, 2, 1, 16), 3.0)                           # fits the scale there is
    assert not OK.write(c, small, [5], [2])
    assert c.scale[0, 0, 0] == 1.0 and np.all(c.values(0, 5) == 3.0) and np.all(c.values(0, 4) == 1.0)
    assert OK.write(c, np.full((1, 1, 1, 16), np.nan), [7], [1]) and c.scale[0, 0, 0] == 1.0


def test_tokens_away_have_no_part_in_the_scale():
    c = _cache([2, -1], 8, 8, 4)
    x = np.full((1, 8, 1, 16), 2.0)
    x[0, 4:] = 1e6
    assert OK.write(c, x, [0], [8])
    assert c.scale[0, 0, 0] == 2.0 ** -7 and np.all(c.values(0, 3) == 2.0)
    c = _cache([-1, 2], 8, 4, 4)                                  # a page of its own: nothing of it changes
    assert OK.write(c, x, [0], [4])
    assert c.scale[0, 0, 0] == 1.0


def test_negative_start_skips_the_sequence():
    c = _cache([2, 3], 8, 4, 4)
    before = c.rows.copy()
    assert OK.write(c, np.ones((1, 6, 1, 16)), [-2], [6])
    assert np.array_equal(c.rows, before) and np.all(c.scale == 1.0)
