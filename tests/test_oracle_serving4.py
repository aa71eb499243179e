"""Pins of oracle/serving.py's 4-bit rows, bounds of pages and their selection (no GPU needed)."""
import numpy as np

from oracle import serving as S


def test_four_bit_values_and_ties():
    ints, scales, byte = S.quantise_row4([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [0.0] * 8)
    assert byte == 127 + 2 - 9
    assert S.row_values4(ints, scales, byte)[:8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert S.pack4([1, 2, 15, 0]).tolist() == [0x21, 0x0F]


def test_four_bit_rows_are_near():
    """The largest of 16 is within half an 8-bit step (2^-4) of its scale's; others within half a step of theirs, 1/6 of that largest."""
    rng = np.random.default_rng(1)
    for _ in range(20):
        x = rng.standard_normal(64) * np.exp(rng.standard_normal(64))
        c, s, byte = S.quantise_row4(x)
        y = S.row_values4(c, s, byte)
        big = np.repeat(np.abs(x).reshape(-1, 16).max(1), 16)
        assert np.all(np.abs(y - x) <= big * (1 / 6 * (1 + 2.0 ** -4) + 2.0 ** -4))
        assert np.array_equal(S.row_values4(*S.quantise_row4(y)), y) or np.abs(S.row_values4(*S.quantise_row4(y)) - y).max() <= big.max() / 6


def test_four_bit_specials():
    assert S.quantise_row4(np.zeros(16))[2] == 127 and not S.quantise_row4(np.zeros(16))[1].any()
    c, s, byte = S.quantise_row4([np.inf, -1.0] + [0.5] * 14 + [np.nan] + [1.0] * 15 + [1.0] * 16)
    v = S.row_values4(c, s, byte)
    assert byte == 127 - 9 and v[0] == 2688 * 2.0 ** -9 and np.isnan(v[16:32]).all() and np.all(np.abs(v[32:] - 1.0) <= 2.0 ** -4)
    assert S.quantise_row4(np.full(16, 1e-300))[2] == 127 + S.MIN_EXP
    # a row that is turned keeps the power of two it had before
    assert S.quantise_row4([1.4] * 16, before=[1.0] * 16)[2] == 127 - 9 and S.quantise_row4([1.4] * 16, before=[1.0] * 16, more=3)[2] == 127 - 6


def test_bounds_hold_every_key():
    rng = np.random.default_rng(2)
    k = rng.standard_normal((7, 24)) * np.exp(2 * rng.standard_normal(24))
    codes, byte = S.page_bounds(k)
    lo, hi = codes * 2.0 ** (byte - 127)
    assert np.all(lo <= k.min(0)) and np.all(hi >= k.max(0)) and np.abs(codes).max() <= 127 and np.abs(codes).max() >= 63
    assert S.page_bounds(np.full((2, 8), 127.0))[1] == 127 and S.page_bounds(np.full((2, 8), 127.1))[1] == 128
    assert S.page_bounds(np.zeros((1, 8)))[1] == 127 and not S.page_bounds(np.zeros((1, 8)))[0].any()
    codes, byte = S.page_bounds(np.array([[np.nan, np.inf, 1.0], [np.nan, -np.inf, np.nan]]))
    assert codes.tolist() == [[0, -127, 64], [0, 127, 64]] and byte == 127 - 6


def test_scores_are_no_less_than_any_keys():
    rng = np.random.default_rng(3)
    k, qs = rng.standard_normal((9, 16)), rng.standard_normal((3, 16))
    score = S.page_score(qs, *S.page_bounds(k))
    rounded = [i * 2.0 ** e for i, e in map(S.query_integers, qs)]
    assert score >= max(float(q @ x) for q in rounded for x in k)


def test_selection():
    assert S.select_pages([5.0, 1.0, 9.0, 9.0, 2.0, 9.0], 3, 0, 0) == [2, 3, 5]
    assert S.select_pages([5.0, 1.0, 9.0, 9.0, 2.0, 9.0], 2, 0, 0) == [2, 3]
    assert S.select_pages([5.0, 1.0, 9.0, 9.0, 2.0, 9.0], 3, 1, 1) == [0, 2, 5]
    assert S.select_pages([1.0, None, -5.0], 2, 0, 0) == [0, 2] and S.select_pages([1.0, None], 5, 1, 1) == [0, 1]


def test_touched_pages():
    assert S.touched_pages([5, 0, 9], None, 4, 100) == {(0, 1): 1, (2, 2): 1}
    assert S.touched_pages([5, 9], [0, 2, 2], 4, 100) == {(0, 0): 4, (0, 1): 1}
    assert S.touched_pages([50], [0, 3], 4, 8) == {}
