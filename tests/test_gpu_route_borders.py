"""mxmoe_route on an MI355X where FP32 and FP64 disagree. Ids and weights
against the float64 oracle, within the router tests' bounds."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def _check(dv, rows, top_k, **kw):
    from test_gpu_route import _check as check

    bias = kw.pop("bias", None)
    if bias is not None:
        bias = torch.tensor(bias, dtype=torch.float32, device="cuda")
    return check(dv, torch.as_tensor(np.asarray(rows, dtype=np.float32)).cuda(), top_k, bias, **kw)


def _rising(start, count):
    """FP32 neighbours from start on."""
    v = [np.float32(start)]
    while len(v) < count:
        v.append(np.nextafter(v[-1], np.float32(np.inf)))
    return np.array(v, dtype=np.float32)


STARTS = (12.0, 16.0, 20.0, 22.5, 23.5, 24.0, 25.0, 26.0, 28.0, 29.0, 29.9, 29.9999)


@pytest.mark.parametrize("experts", [24, 64, 200])
def test_equal_sigmoids_of_different_logits(dv, experts):
    """Neighbouring logits, the larger at the higher index: from about 22.8 on
    their FP64 sigmoids are equal, and the lowest index is chosen."""
    rng = np.random.default_rng(experts)
    x = rng.standard_normal((len(STARTS), experts)).astype(np.float32)
    for row, start in zip(x, STARTS):
        row[np.sort(rng.choice(experts, 12, replace=False))] = _rising(start, 12)
    _check(dv, x, 6, score="sigmoid")
    _check(dv, x, 1, score="sigmoid")
    _check(dv, [[25.0, 25.000002], [28.0, 28.0001], [29.0, 29.0009]], 1, score="sigmoid")


@pytest.mark.parametrize("per", [1, 2, 3, 16])
def test_equal_group_scores_of_different_logits(dv, per):
    """A group's best logit above the next group's by one FP32 step."""
    rng = np.random.default_rng(per)
    x = rng.standard_normal((len(STARTS), 12 * per)).astype(np.float32)
    for row, start in zip(x, STARTS):
        row[np.arange(12) * per + rng.integers(0, per, 12)] = _rising(start, 12)
    for best in (1, 2):
        _check(dv, x, 2, score="sigmoid", groups=12, top_groups=3, group_best=best)
        _check(dv, x, 1, score="sigmoid", groups=12, top_groups=1, group_best=best)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tiny_logits_are_equal(dv, score):
    """Logits so small that FP64 scores do not tell them apart, whatever else is
    in the row."""
    tiny = [0.0, 1e-20, 2e-20, -1e-20, 1e-38, -1e-30, 3e-20, 2e-22]
    rows = [tiny, tiny[::-1], [1.0, *tiny[1:]], [1.0, *tiny[1:7], -750.0],
            [-3.0, 4e-21, *tiny[2:]], [0.0, 1e-20, -2.0, -2.0, -2.0, -2.0, -2.0, -2.0]]
    for k in (1, 2, 5, 8):
        _check(dv, rows, k, score=score)
    for groups in (2, 4):
        _check(dv, rows, 1, score=score, groups=groups, top_groups=1)
        _check(dv, rows, 2, score=score, groups=groups, top_groups=2)


def test_small_differences_that_count(dv):
    """FP32 neighbours whose FP64 scores differ keep the larger first."""
    x = np.stack([_rising(s, 16) for s in (-40.0, -1.0, -1e-3, 1e-3, 0.5, 3.0, 10.0)])
    for score in ("softmax", "sigmoid"):
        _check(dv, x, 5, score=score)
        _check(dv, x, 5, score=score, groups=4, top_groups=2)


def test_group_scores_that_cancel(dv):
    """Two large biases of opposite sign in a group: the score is the small rest,
    which FP32 sums lose."""
    x = np.random.default_rng(3).standard_normal((256, 16)).astype(np.float32)
    for big in (1e3, 1e5, 1e6):
        for groups in (2, 3, 8):
            bias = [big, -big] * groups
            for score in ("sigmoid", "softmax"):
                _check(dv, x[:, : 2 * groups], 1, bias=bias, score=score, groups=groups,
                       top_groups=1, group_best=2)


@pytest.mark.parametrize("scale", [1.0, 2.5, 1e30])
def test_weights_of_small_scores(dv, scale):
    """Chosen scores below FP32's range: renormalised weights are those of the
    formula, and so is a product with a large scale."""
    rows = [[-95, -96, -97, -98, -200, -300], [-60, -61, -120, -300, -699, -699],
            [-500.5, -500, -501, -502, -503, -700], [-90, -103.5, -104, -88, -89, -87.5],
            [-64, -65, -63, -66, -80, -81], [-707, -706, -706.5, -900, -1e30, -800]]
    for k in (1, 2, 5):
        _check(dv, rows, k, score="sigmoid", renormalize=True, scale=scale)
        _check(dv, rows, k, score="sigmoid", scale=scale)
    rows = [[0, -110, -110, -112, -90, -50], [3, -100, -101, -102, -103, -103.5],
            [0, -650, -651, -650.25, -700, -705], [5, 5, -60, -59, -61, -62]]
    bias = [0, 3, 2.5, 2.25, 2, 1.75]
    for k in (1, 2, 5, 6):
        _check(dv, rows, k, bias=bias, renormalize=True, scale=scale)
        _check(dv, rows, k, bias=bias, scale=scale)


def test_weights_of_zero_scores(dv):
    """A score below 2^-1022 is zero, and a sum of zero leaves the weights zero."""
    bias = [0, 3, 2, 0]
    ids, w = _check(dv, [[0, -800, -900, -1e30]], 2, bias=bias, renormalize=True)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[0, 0]]
    ids, w = _check(dv, [[-800, -900, -750, -1e30]], 2, score="sigmoid", renormalize=True)
    assert w.tolist() == [[0, 0]]
    _check(dv, [[0, -800, -700, -1e30]], 2, bias=bias, renormalize=True)
