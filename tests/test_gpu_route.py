"""mxmoe_route on an MI355X against the float64 oracle: ids equal, weights
within FP32 arithmetic.

The weight bound: softmax's exp(l - max) has the rounded argument's error,
2^-24 |l - max|, and 2 ulp of its own; a sum over at most 1024 terms (16 in a
lane, 6 exchanges) adds 22 roundings; the division, the product with the scale
and a renormalisation (its sum, its division) stay below 20 more. In units of
2^-24, relative: 64 + |l - max|, doubled where the weights are renormalised.
Weights below FP32's normal range are held to 2^-126."""

import sys

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


def _check(dv, logits, top_k, bias=None, **kw):
    from oracle import decode

    print(f"route {tuple(logits.shape)} {logits.dtype} k={top_k} {kw}", flush=True)
    sys.stdout.flush()
    ids, w = dv.route(logits, top_k, bias=bias, **kw)
    torch.cuda.synchronize()
    values = logits.double().cpu().numpy()
    want_ids, want = decode.route(values, top_k, bias=None if bias is None else bias.cpu().numpy(),
                                  **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    finite = np.where(np.isfinite(values), values, 0.0)
    span = np.abs(finite - finite.max(1, keepdims=True)).max(1, keepdims=True)
    tol = 2.0**-24 * (64 + span) * (2 if kw.get("renormalize") else 1)
    got = w.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol * np.abs(want) + 2.0**-126), np.abs(got - want).max()
    return ids, w


def _logits(seed, t, e, dtype=torch.float32, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(t, e, generator=g, device="cuda")).to(dtype)


def _bias(seed, e):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 0.1 * torch.randn(e, generator=g, device="cuda")


@pytest.mark.parametrize("t,e,k,kw", [
    (1, 1, 1, dict()), (3, 2, 2, dict(renormalize=True)), (8, 256, 8, dict(score="sigmoid")),
    (5, 60, 4, dict()), (7, 65, 6, dict(renormalize=True, scale=2.5)), (9, 64, 32, dict()),
    (33, 128, 8, dict(score="sigmoid", renormalize=True)), (130, 384, 8, dict()),
    (4, 1024, 32, dict(renormalize=True)), (6, 1000, 10, dict(score="sigmoid")),
    (16, 256, 8, dict(groups=8, top_groups=4, group_best=1)),
    (16, 256, 8, dict(groups=8, top_groups=4, group_best=2, score="sigmoid", renormalize=True)),
    (16, 256, 8, dict(groups=8, top_groups=8, group_best=2)),
    (5, 60, 5, dict(groups=12, top_groups=1, group_best=2, renormalize=True)),
    (5, 64, 3, dict(groups=64, top_groups=3, group_best=2)),
    (5, 96, 7, dict(groups=3, top_groups=2, group_best=2, score="sigmoid")),
    (5, 1024, 9, dict(groups=2, top_groups=1, group_best=2, score="sigmoid")),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
def test_route(dv, t, e, k, kw, dtype, biased):
    _check(dv, _logits(t * 1000 + e, t, e, dtype), k, _bias(e, e) if biased else None, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(score="sigmoid"), dict(groups=8, top_groups=3),
                                dict(groups=8, top_groups=3, group_best=2, score="sigmoid")])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lowest_index(dv, kw, biased):
    """Few distinct logits: most choices and group scores are equal."""
    g = torch.Generator(device="cuda").manual_seed(7)
    logits = torch.randint(0, 3, (40, 128), generator=g, device="cuda").float()
    bias = torch.randint(0, 2, (128,), generator=g, device="cuda").float() if biased else None
    _check(dv, logits, 9, bias, **kw)
    _check(dv, torch.zeros(2, 128, device="cuda"), 9, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_experts(dv, score, groups, biased):
    """-infinity and NaN take an expert out; rows with few or none left; the
    type's lowest value is a logit like any other; +infinity and saturated
    scores."""
    x = _logits(3, 12, 64)
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x[0] = -inf
    x[1] = float("nan")
    x[2, 1:] = -inf
    x[3, :62] = float("nan")
    x[4, 10:40] = -inf
    x[5] = low
    x[6, 5:] = low
    x[7, 3] = inf
    x[8, 3:9] = inf
    x[9, 20:] = -200.0
    x[10] *= 20  # sigmoids that round to one, next to some that do not
    x[11, :16] = -inf
    _check(dv, x, 6, _bias(1, 64) if biased else None, score=score, groups=groups,
           top_groups=max(1, groups // 2), group_best=2, renormalize=True)
    _check(dv, x, 6, _bias(1, 64) if biased else None, score=score, groups=groups,
           top_groups=max(1, groups // 2))


def test_strided_rows_and_given_outputs(dv):
    """Rows at any stride and element offset; what lies past the outputs stays."""
    full = _logits(11, 9, 101, torch.bfloat16)
    view = full[:, 1:78]
    ids, w = _check(dv, view, 5)
    again_i = torch.full((11, 5), 77, dtype=torch.int32, device="cuda")
    again_w = torch.full((11, 5), 77.0, device="cuda")
    dv.route(view, 5, ids=again_i[1:10], weights=again_w[1:10])
    assert torch.equal(again_i[1:10], ids) and torch.equal(again_w[1:10], w)
    assert (again_i[[0, 10]] == 77).all() and (again_w[[0, 10]] == 77).all()
    _check(dv, _logits(12, 18, 77)[::2], 5)


def test_many_rows(dv):
    """A prefill's rows, the grouped sigmoid choice with a bias."""
    _check(dv, _logits(21, 2051, 256), 8, _bias(4, 256), score="sigmoid", groups=8, top_groups=4,
           group_best=2, renormalize=True, scale=2.5)


def test_refusals(dv):
    x = _logits(1, 4, 64)
    for bad in (dict(top_k=0), dict(top_k=33), dict(groups=5), dict(groups=8, top_groups=9),
                dict(group_best=3), dict(score="relu"), dict(bias=_bias(1, 63)),
                dict(ids=torch.empty(4, 3, dtype=torch.int32, device="cuda")),
                dict(weights=torch.empty(4, 4, dtype=torch.float64, device="cuda"))):
        with pytest.raises(ValueError):
            dv.route(x, **{"top_k": 4, **bad})
    with pytest.raises(ValueError):
        dv.route(x.double(), 4)
    with pytest.raises(ValueError):
        dv.route(x.t(), 4)


def test_odd_biases(dv):
    """Biases of infinity and NaN, and large ones, whose FP32 sums lose the score."""
    x = _logits(31, 6, 96)
    bias = _bias(5, 96)
    bias[3], bias[4], bias[50] = float("-inf"), float("nan"), float("inf")
    for score in ("softmax", "sigmoid"):
        ids, _ = dv.route(x, 8, score=score, bias=bias, groups=3, top_groups=2, group_best=2)
        ids = ids.cpu()
        assert (ids[:, 0] == 50).all() and not torch.isin(ids, torch.tensor([3, 4])).any()
    _check(dv, x, 8, 1e6 + 0.25 * torch.arange(96, device="cuda") % 3, score="sigmoid")


def test_on_a_given_stream(dv):
    """Another stream than the current one, outputs of its own."""
    x = _logits(41, 64, 256)
    want = dv.route(x, 8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = dv.route(x, 8, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured(dv):
    """Replays with other logits, eager calls between."""
    x, ids, w = _logits(51, 17, 72), *(torch.empty(17, 6, dtype=t, device="cuda")
                                       for t in (torch.int32, torch.float32))
    kw = dict(score="sigmoid", bias=_bias(7, 72), groups=9, top_groups=4, group_best=2)
    dv.route(x, 6, ids=ids, weights=w, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dv.route(x, 6, ids=ids, weights=w, **kw)
    for seed in range(4):
        x.copy_(_logits(60 + seed, 17, 72))
        graph.replay()
        torch.cuda.synchronize()
        want = dv.route(x, 6, **kw)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])


def test_most_rows(dv):
    """2^24 rows: the last ones, and a sample of the others."""
    t = 1 << 24
    logits = torch.randn(t, 2, device="cuda")
    ids, weights = dv.route(logits, 1)
    best = logits.argmax(1)
    assert torch.equal(ids[:, 0].long(), best)
    want = torch.softmax(logits.double(), 1).amax(1)
    # (FP32: exp, sum and quotient, a few halves of 2^-23 each.)
    assert ((weights[:, 0].double() - want).abs() <= 2.0 ** -20 * want).all()
