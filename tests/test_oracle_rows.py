"""The oracle of MXFP4 and the products of any number of rows against hand-worked values and brute force (CPU)."""

import math

import numpy as np
import pytest

from oracle import rows


def test_e2m1_values():
    assert [rows.e2m1_value(c) for c in range(8)] == [0, 0.5, 1, 1.5, 2, 3, 4, 6] == list(rows.E2M1)
    assert [rows.e2m1_value(c) for c in range(8, 16)] == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    assert math.copysign(1, rows.e2m1_value(8)) == -1


def test_ties_go_to_the_even_code():
    for y, code in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)):
        assert rows.e2m1_round(y) == code and rows.e2m1_round(-y) == code | 8
        assert rows.E2M1[rows.e2m1_round(np.nextafter(y, 9))] > y > rows.E2M1[rows.e2m1_round(np.nextafter(y, 0))]
    assert rows.e2m1_round(-0.0) == 8 and rows.e2m1_round(6.0) == 7
    with pytest.raises(ValueError):
        rows.e2m1_round(6.01)


def test_the_smallest_exponent():
    for amax, e in ((6.0, 0), (np.nextafter(6.0, 7), 1), (3.0, -1), (12.0, 1), (1.0, -2), (0.75, -3), (0.0, -127),
                    (2.0**-140, -127), (2.0**127, 125), (3.4e38, 126)):
        assert rows.fp4_exponent(float(amax)) == e


def test_a_hand_worked_block():
    v = np.zeros((1, 64))
    v[0, :6] = [12, -5, 0.4, -0.5, 0.6, 10.1]   # e = 1: halves 6, -2.5, .2, -.25, .3, 5.05
    v[0, 32] = np.nan
    v[0, 33] = -1
    codes, scales = rows.quantize4(v)
    assert scales.tolist() == [[128, 255]]
    assert codes[0, :3].tolist() == [7 | 12 << 4, 0 | 8 << 4, 1 | 7 << 4]
    assert codes[0, 16] == 7 | 15 << 4 and codes[0, 17] == 7 | 7 << 4
    back = rows.values(codes, scales)
    assert back[0, :6].tolist() == [12, -4, 0, 0, 1, 12] and np.isnan(back[0, 32:]).all()


def test_products_against_loops():
    rng = np.random.default_rng(3)
    w, x = rng.integers(0, 256, (2, 4, 32), dtype=np.uint8), rng.integers(0, 256, (5, 32), dtype=np.uint8)
    ws, xs = rng.integers(120, 130, (2, 4, 2), dtype=np.uint8), rng.integers(120, 130, (5, 2), dtype=np.uint8)
    table = [0, .5, 1, 1.5, 2, 3, 4, 6]

    def value(b, s, k):
        c = int(b[k // 2]) >> 4 * (k % 2) & 15
        return (-1 if c > 7 else 1) * table[c % 8] * 2.0 ** (int(s[k // 32]) - 127)

    offsets, order = np.array([0, 1, 4]), np.array([3, 9, 0, 6, 1])
    got, slack, written = rows.grouped(w, ws, x, xs, offsets, order, gather=2, rows=5)
    assert written.tolist() == [True] * 4 + [False] and (slack[:4] > 0).all()
    for i, e in enumerate([0, 1, 1, 1]):
        for n in range(4):
            want = sum(value(w[e, n], ws[e, n], k) * value(x[order[i] // 2], xs[order[i] // 2], k) for k in range(64))
            assert got[i, n] == want
    plain, _, _ = rows.grouped(w, ws, x, xs, offsets)
    assert np.array_equal(plain[0], rows.product(w[0], ws[0], x[:1], xs[:1])[0][0])
    z, _ = rows.product(w[0], ws[0], x, xs)
    h, _ = rows.product(w[0], ws[0], x, xs, gated=True)
    assert np.allclose(h, z[:, :2] / (1 + np.exp(-z[:, :2])) * z[:, 2:], rtol=1e-14)


def test_sort_and_combine():
    ids = np.array([[1, 0], [3, 1], [-1, 0], [1, 2]], dtype=np.int32)
    order, offsets = rows.sort_pairs(ids, 3)
    assert order.tolist() == [1, 5, 0, 3, 6, 7, 2, 4] and offsets.tolist() == [0, 2, 5, 6]
    y = np.arange(16.0).reshape(4, 2, 2)
    w = np.array([[1, 2], [3, 4], [5, 6], [7, 8]], dtype=np.float32)
    out, slack = rows.combine(y, ids, w, 3)
    assert out.tolist() == [[4, 7], [24, 28], [60, 66], [7 * 12 + 8 * 14, 7 * 13 + 8 * 15]] and slack.shape == (4, 2)


def test_a_planted_mistake_is_outside_the_bounds():
    """Scales of the neighbouring block, and codes in the other half of a byte, are no rounding."""
    rng = np.random.default_rng(5)
    w, x = rng.integers(0, 256, (8, 64), dtype=np.uint8), rng.integers(0, 256, (8, 64), dtype=np.uint8)
    ws, xs = rng.integers(120, 130, (8, 4), dtype=np.uint8), rng.integers(120, 130, (8, 4), dtype=np.uint8)
    exact, slack = rows.product(w, ws, x, xs)
    bound = rows.bf16_bound(exact, slack)
    for other in (rows.product(w, np.roll(ws, 1, 1), x, xs)[0], rows.product(w << 4 | w >> 4, ws, x, xs)[0]):
        assert (np.abs(other - exact) > bound).mean() > 0.9
