"""The sums of products of any number of rows on an MI355X, of MXFP8 rows above all: FP32 keeps what lies 2^-14 below the largest product beside it, as
mxgemm and mxmoe_experts do, for any number of rows and by every kernel. Inputs whose large products cancel leave results
made of small ones alone; every partial sum of them is an FP32 value in any order, so that the results are the exact sums,
rounded once to BF16."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle, tolerance  # noqa: E402
from rows_cases import close, cuda, f64, weights  # noqa: E402

W_FORMS = ["mxfp4", "mxfp8"]


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def _cancelling(rng, w_form, rows, n, k, experts=1):
    """W (codes, scales) [experts, n, k] and x [rows, k]: in each 32 of K one product of 16, its sign the other one in the
    next 32, and 31 products of 1 to 6 times 2^-10. Sums are multiples of 2^-10 up to 16 k / 32 <= 2^13: 23 bits. Each row
    has a power of two of its own."""
    at = 32 * np.arange(k // 32) + rng.integers(0, 32, k // 32)
    one, half, four, sign = (2, 1, 6, 8) if w_form == "mxfp4" else (0x38, 0x30, 0x48, 0x80)
    w = np.where(rng.random((experts, n, k)) < 0.5, one, half).astype(np.uint8)
    turn = (np.arange(k // 32) + rng.integers(0, 2, (experts, n, 1))) % 2
    w[..., at] = four | sign * turn
    x = rng.integers(1, 4, (rows, k), dtype=np.uint8)  # 2^-9 times 1 to 3
    x[:, at] = 0x48
    ws = np.broadcast_to(rng.integers(120, 135, (experts, n, 1), dtype=np.uint8), (experts, n, k // 32)).copy()
    xs = np.broadcast_to(rng.integers(120, 135, (rows, 1), dtype=np.uint8), (rows, k // 32)).copy()
    return (oracle.pack4(w) if w_form == "mxfp4" else w, ws), (x, xs)


def _rounded(exact):
    return torch.from_numpy(exact).bfloat16().cuda()


# (rows, n, k): streams of 1 to 32 rows, K divided among workgroups, tiles alone on a CU and by two, whole and not.
SIZES = [(1, 40, 128), (7, 264, 2048), (24, 264, 640), (33, 136, 4096), (40, 264, 16384), (130, 520, 8320),
         (289, 1032, 640), (1100, 4104, 384), (2060, 4104, 256)]


@pytest.mark.parametrize("w_form", W_FORMS)
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_small_products_beside_large_ones_that_cancel(dv, w_form, rows, n, k):
    (w, ws), x = _cancelling(np.random.default_rng(rows + n + k), w_form, rows, n, k)
    got = dv.Linear(cuda(w[0]), cuda(ws[0]))(*map(cuda, x))
    assert torch.equal(got, _rounded(oracle.product(w[0], ws[0], *x)[0]))


@pytest.mark.parametrize("form", ["gather", "scatter"])
@pytest.mark.parametrize("groups,k", [([3, 0, 1, 9, 2], 2304), ([40, 0, 131, 300], 640)])
@pytest.mark.parametrize("w_form", W_FORMS)
def test_experts(dv, w_form, groups, k, form):
    rng = np.random.default_rng(len(groups) + k)
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    rows = int(offsets[-1]) + int(offsets[-1]) % 2
    order = rng.permutation(rows).astype(np.int32)
    gather, scatter = (2, False) if form == "gather" else (0, True)
    w, x = _cancelling(rng, w_form, rows // 2 if gather else rows, 136, k, len(groups))
    got = dv.GroupedLinear(*map(cuda, w))(*map(cuda, x), cuda(offsets), cuda(order), gather, scatter)
    exact, _, written = oracle.grouped(*w, *x, offsets, order, gather, scatter, rows=rows)
    assert torch.equal(got[cuda(written)], _rounded(exact)[cuda(written)])


@pytest.mark.parametrize("w_form,x_form", [("mxfp4", "mxfp8"), ("mxfp8", "mxfp8"), ("mxfp4", "mxfp4")])
@pytest.mark.parametrize("rows,n,k", [(2, 128, 2048), (70, 320, 4096), (130, 576, 8320), (300, 1088, 1152),
                                      (1100, 4160, 512), (2060, 4160, 1152)])
def test_the_bound_of_the_decode_projection(dv, w_form, x_form, rows, n, k):
    """Random operands: within a BF16 step and 1e-6 of the sum of magnitudes (a gated row's gate and up each)."""
    rng = np.random.default_rng(rows * n + k)
    w, x = weights(rng, w_form, n, k), weights(rng, x_form, rows, k)
    w[1][...] += rng.integers(0, 3, w[1].shape, dtype=np.uint8)
    args = *map(cuda, w), *map(cuda, x)
    exact = oracle.product(*w, *x)[0]
    total = np.abs(oracle.values(*x)) @ np.abs(oracle.values(*w)).T
    got = dv.Linear(*args[:2])(*args[2:])
    assert tolerance.within(got.view(torch.int16).cpu().numpy().view(np.uint16), exact, total)
    got = f64(dv.Linear(*args[:2], gated=True)(*args[2:]))
    g, u, d = exact[:, : n // 2], exact[:, n // 2:], tolerance.REL_ABS_SUM * total
    silu = g / (1 + np.exp(-g))
    slack = (oracle.SILU_SLOPE * d[:, : n // 2] * (np.abs(u) + d[:, n // 2:]) + np.abs(silu) * d[:, n // 2:]
             + oracle.GATE_ROUNDING * (10 + np.abs(g)) * np.abs(silu * u))
    assert (np.abs(got - silu * u) <= oracle.bf16_bound(silu * u, slack)).all()


@pytest.mark.parametrize("rows", [2, 300])
@pytest.mark.parametrize("w_form", W_FORMS)
def test_rows_of_zeros_beside_them(dv, w_form, rows):
    """Zeros quantize to scale byte 0: they cost the rows beside them no bits."""
    (w, ws), (x, xs) = _cancelling(np.random.default_rng(rows), w_form, rows, 136, 2048)
    x[1::3], xs[1::3] = 0, 0
    x[0, 64:96], xs[0, 2] = 0, 0
    w[0, 5], ws[0, 5] = 0, 0
    got = dv.Linear(cuda(w[0]), cuda(ws[0]))(*map(cuda, (x, xs)))
    assert torch.equal(got, _rounded(oracle.product(w[0], ws[0], x, xs)[0]))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("w_form,scales", [("mxfp4", (0, 1, 2)), ("mxfp8", (0, 1, 2)), ("mxfp4", (247, 250)),
                                           ("mxfp8", (247, 250)), ("mxfp4", None), ("mxfp8", None)])
@pytest.mark.parametrize("rows", [3, 40, 200])
def test_values_that_bf16_does_not_hold(dv, rows, w_form, scales, gated):
    """Scale bytes outside 3..246 in some blocks of W (x has scales that bring the products back) or, without such ones, of
    x: e4m3 codes down to 2^-9 below them. Within the oracle's bound, that of the scaled instruction there; infinities of
    partial sums would show."""
    n, k = 192, 1408
    rng = np.random.default_rng(rows + len(w_form) + (scales or (7,))[0])
    w, x = weights(rng, w_form, n, k), weights(rng, "mxfp8", rows, k)
    if w_form == "mxfp8":
        w[0][...] = rng.integers(0, 256, w[0].shape, dtype=np.uint8) & 0xBF  # up to 1.875, subnormals among them
    x[0][...] = rng.integers(0, 256, x[0].shape, dtype=np.uint8) & 0xBF
    odd, other = (w, x) if scales else (x, w)
    low = scales is None or scales[0] < 9
    odd[1][...] = rng.integers(3, 9, odd[1].shape) if low else rng.integers(240, 247, odd[1].shape)
    some = rng.random(odd[1].shape) < 0.05
    odd[1][some] = rng.choice(scales or (0, 1, 2), int(some.sum()))
    other[1][...] = rng.integers(236, 244, other[1].shape) if low else rng.integers(10, 16, other[1].shape)
    assert oracle.leaves_bf16(oracle.values(*odd), odd[1])
    lin = dv.Linear(*map(cuda, w), gated=gated)
    with np.errstate(over="ignore"):  # (the oracle's exp of a large negative gate)
        assert close(lin(*map(cuda, x)), *oracle.product(*w, *x, gated=gated))


@pytest.mark.parametrize("rows", [3, 40, 200])
@pytest.mark.parametrize("low", [True, False])
@pytest.mark.parametrize("w_form", W_FORMS)
def test_values_at_the_ends_of_what_bf16_holds(dv, rows, low, w_form):
    """Scale bytes 3..8, where e4m3 codes are BF16 subnormals, and 240..246: no bit is lost, by W or by x."""
    n, k = 192, 1408
    rng = np.random.default_rng(rows + len(w_form))
    w, x = weights(rng, w_form, n, k), weights(rng, "mxfp8", rows, k)
    if w_form == "mxfp8":
        w[0][...] = rng.integers(0, 256, w[0].shape, dtype=np.uint8) & 0xBF
    x[0][...] = rng.integers(0, 256, x[0].shape, dtype=np.uint8) & 0xBF
    for odd, other in ((w, x), (x, w)):
        odd[1][...] = rng.integers(3, 9, odd[1].shape) if low else rng.integers(240, 247, odd[1].shape)
        other[1][...] = rng.integers(236, 244, other[1].shape) if low else rng.integers(10, 16, other[1].shape)
        got = dv.Linear(*map(cuda, w))(*map(cuda, x))
        total = np.abs(oracle.values(*x)) @ np.abs(oracle.values(*w)).T
        assert tolerance.within(got.view(torch.int16).cpu().numpy().view(np.uint16), oracle.product(*w, *x)[0], total)


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("w_form", W_FORMS)
def test_nan_codes_stay_in_their_rows_and_columns(dv, rows, w_form):
    rng = np.random.default_rng(rows)
    w, x = weights(rng, w_form, 136, 640), weights(rng, "mxfp8", rows, 640)
    x[0][1, 333] = 0x7F
    x[1][2, 7] = 255
    if w_form == "mxfp8":
        w[0][70, 2] = 0xFF
    w[1][9, 0] = 255
    got = dv.Linear(*map(cuda, w))(*map(cuda, x))
    want = torch.from_numpy(oracle.product(*w, *x)[0]).cuda()
    assert torch.equal(got.isnan(), want.isnan()) and got[1:3].isnan().all() and not got[3:, 10:70].isnan().any()


@pytest.mark.parametrize("rows,n,k", [(7, 264, 2048), (130, 520, 8320), (300, 1032, 640)])
@pytest.mark.parametrize("w_form", W_FORMS)
def test_captured_with_values_that_come_to_leave_bf16(dv, w_form, rows, n, k):
    """One graph, replayed on rows that BF16 holds, that it does not hold, and again that it holds, with eager work and a
    call on another stream between: the eager results each time."""
    rng = np.random.default_rng(rows)
    lin = dv.Linear(*map(cuda, weights(rng, w_form, n, k)))
    inputs = [weights(rng, "mxfp8", rows, k) for _ in range(3)]
    inputs[1][1][::2, 3] = 1                              # (rows scaled by 2^-126 in one block)
    inputs[1][1][1, 5] = 255
    x, xs = map(cuda, inputs[0])
    lin(x, xs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lin(x, xs)
    side = torch.cuda.Stream()
    for i in (0, 1, 2, 1, 0):
        x.copy_(cuda(inputs[i][0]))
        xs.copy_(cuda(inputs[i][1]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = lin(x, xs)
        other = lin(x, xs, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(other.view(torch.int16), want.view(torch.int16))
        assert bool(want.isnan().any()) == (i == 1)
