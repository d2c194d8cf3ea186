"""The oracle of 8-bit pages, of the pages' weights and of eviction, pinned by
hand-made cases (no GPU)."""

import numpy as np

from oracle import cache as OC


def test_codes_are_e4m3():
    """Against the format's definition: sign, four exponent bits of bias 7,
    three of the magnitude, subnormals, no infinities."""
    for c in range(128):
        e, m = c >> 3, c & 7
        want = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if c == 127:
            assert np.isnan(OC.values8(np.uint8(c)))
        else:
            assert OC.values8(np.uint8(c)) == want and OC.values8(np.uint8(c | 128)) == -want
            assert OC.codes8(want) == c and OC.codes8(-want) == c | 128
    assert OC.codes8(448.0) == 126 and OC.codes8(1e30) == 126 and OC.codes8(np.nan) & 127 == 127


def test_ties_go_to_the_even_code():
    v = OC.E4M3[:127]
    mid = (v[1:] + v[:-1]) / 2
    c = OC.codes8(mid)
    assert np.all(c % 2 == 0) and np.all(np.abs(c.astype(int) - (np.arange(126) + 0.5)) == 0.5)
    eps = np.spacing(mid)
    assert np.array_equal(OC.codes8(mid - eps), np.arange(126)) and np.array_equal(OC.codes8(mid + eps), np.arange(1, 127))


def test_a_block_grows_and_forgets_nothing_above():
    """A larger token raises the scale; what is there is rounded again: exact
    but for what falls among the subnormals."""
    rows = OC.Rows8(2)
    rows.append(0, np.array([[1.0, 3.0], [448.0, -7.0]]))
    assert rows.e == [0] and np.array_equal(rows.values(), [[1, 3], [448, -7]])
    rows.append(2, np.array([[449.0, 0.0]]))
    assert rows.e == [1] and np.array_equal(rows.values()[:2], [[1, 3], [448, -7]])
    rows.append(2, np.array([[448.0 * 2 ** 12, 0.0]]))                # rolled back, a far larger one
    assert rows.e == [12]
    assert np.array_equal(rows.values()[:2], [[0, 0], [448, -8]])     # 1 and 3 lie below 4, half the least code 8
    rows.append(16 - 13, np.zeros((13, 2)))
    rows.append(16, np.array([[2.0 ** -120, 0.0]]))                   # a new block, its own scale
    assert rows.e == [12, OC.LOW8]


def test_not_finite_is_nan_and_has_no_part_in_the_scale():
    rows = OC.Rows8(3)
    rows.append(0, np.array([[np.inf, 2.0, np.nan]]))
    assert rows.e == [-7] and np.isnan(rows.values()[0, 0]) and rows.values()[0, 1] == 2.0


def test_weights_of_all_pages_sum_to_one_a_row_and_head():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((70, 2, 8))
    q = rng.standard_normal((3, 4, 8))
    pos = np.array([67, 68, 69])
    for window, sinks in ((0, 0), (20, 3)):
        _, lse = OC.attention(q, k, k, pos, 0.3, window, sinks)
        m = OC.weigh(q, lse, k, pos, 0.3, window, sinks, 16)
        assert m.shape == (5,) and abs(m.sum() - 12) < 1e-9
    have = np.ones(70, bool)
    have[16:32] = False
    _, lse = OC.attention(q, k, k, pos, 0.3, 0, 0, have)
    m = OC.weigh(q, lse, k, pos, 0.3, 0, 0, 16, have)
    assert m[1] == 0 and abs(m.sum() - 12) < 1e-9


def test_eviction_by_hand():
    p = OC.Pages(2, 20, 6, 16)
    p.len[:] = [90, 33]                       # six pages, the last of 10 tokens; three
    p.table[0] = [3, 4, 5, 6, 7, 8]
    p.table[1, :3] = [4, 9, 10]
    mass = np.array([[5.0, 1, 1, np.nan, 0, 0], [2.0, 3, 0, 9, 9, 9]])
    assert p.evict(mass, [3, 0], 0, 0) == [3, 2]
    assert p.table[0].tolist() == [3, -2, -2, 6, -2, 8]      # least first, ties by entry; NaN and the open page stay
    assert p.table[1].tolist() == [-2, -2, 10, -1, -1, -1]
    assert mass[0].tolist()[:3] == [5, 0, 0] and mass[1, 0] == 0
    assert p.refs()[[3, 4, 5, 6, 7, 8, 9, 10]].tolist() == [1, 0, 0, 1, 0, 1, 0, 1]
    mass[0, 0] = -1.0
    assert p.evict(mass, [-1, 9], 0, 0) == [0, 0]
    assert p.evict(mass, [0, 0], 1, 27) == [0, 0]            # first token kept; the last 27 reach into page 3
    assert p.evict(mass, [0, 0], 1, 26) == [1, 0]
