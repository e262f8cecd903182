"""Pins of the oracle of the per-row decode operators on cases worked by hand."""

import numpy as np
import pytest

from oracle import decode
from oracle.codecs import bf16_quantum
from workloads import generate


def test_route_softmax_by_hand():
    row = np.log([[0.1, 0.4, 0.2, 0.3]])
    ids, w = decode.route(row, 2)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, [[0.4, 0.3]])
    ids, w = decode.route(row, 2, renormalize=True, scale=2.0)
    assert np.allclose(w, [[8 / 7, 6 / 7]])


def test_route_bias_chooses_but_does_not_weigh():
    ids, w = decode.route(np.zeros((1, 4)), 2, score="sigmoid", bias=[0, 0, 0.5, 0.25])
    assert ids.tolist() == [[2, 3]] and np.allclose(w, 0.5)


def test_route_groups_by_hand():
    # groups {0,1}, {2,3}: best of one favours the second, of two the first
    row = np.array([[1.0, 0.9, 1.1, -5.0]])
    one, _ = decode.route(row, 1, score="sigmoid", groups=2, top_groups=1, group_best=1)
    two, _ = decode.route(row, 2, score="sigmoid", groups=2, top_groups=1, group_best=2)
    assert one.tolist() == [[2]] and two.tolist() == [[0, 1]]


def test_route_ties_and_masks():
    ids, w = decode.route(np.zeros((1, 5)), 3)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 0.2)
    row = np.array([[-np.inf, np.nan, 2.0, -np.inf], [-np.inf] * 4])
    ids, w = decode.route(row, 2, renormalize=True)
    assert ids.tolist() == [[2, -1], [-1, -1]] and w.tolist() == [[1, 0], [0, 0]]


def test_experts_against_a_direct_sum():
    rng = np.random.default_rng(5)
    w13, s13 = zip(*(generate.quantize_mxfp8(rng.standard_normal((64, 64))) for _ in range(3)))
    w2, s2 = zip(*(generate.quantize_mxfp8(rng.standard_normal((64, 32))) for _ in range(3)))
    w13, s13, w2, s2 = (np.stack(v) for v in (w13, s13, w2, s2))
    x = rng.standard_normal((2, 64))
    ids, wt = np.array([[2, 0], [-1, 2]]), np.array([[0.25, 0.75], [1.0, 2.0]])
    got, bound = decode.experts(x, ids, wt, w13, s13, w2, s2)
    val = lambda c, s: decode.dequantize(c, s)  # noqa: E731
    want = np.zeros((2, 64))
    for t, e, w in ((0, 2, 0.25), (0, 0, 0.75), (1, 2, 2.0)):
        z = val(w13[e], s13[e]) @ x[t]
        g = z[:32]
        want[t] += w * (val(w2[e], s2[e]) @ (g / (1 + np.exp(-g)) * z[32:]))
    assert np.allclose(got, want, rtol=1e-12)
    assert (bound >= bf16_quantum(want)).all() and (bound < 0.02 * np.abs(want).max()).all()


def test_adapted_against_a_direct_sum():
    p = generate.random_problem(3, 3, 16, 128)
    rng = np.random.default_rng(6)
    a, b = rng.standard_normal((2, 8, 128)), rng.standard_normal((2, 16, 8))
    x = rng.standard_normal((3, 128))
    got, _ = decode.adapted(x, x, p.w, p.ws, a, b, [0.5, 2.0], [1, -1, 0])
    base = x @ decode.dequantize(p.w, p.ws).T
    want = base + np.stack([2.0 * b[1] @ a[1] @ x[0], np.zeros(16), 0.5 * b[0] @ a[0] @ x[2]])
    assert np.allclose(got, want, rtol=1e-12)


@pytest.mark.parametrize("k", [1, 4])
def test_route_ids_are_distinct(k):
    ids, _ = decode.route(np.random.default_rng(1).standard_normal((50, 9)), k)
    assert all(len(set(r)) == k for r in ids.tolist())
