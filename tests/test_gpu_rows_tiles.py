"""The products of many rows on an MI355X by each of their tiles: small ones alone on a CU and by two, large ones of every
height, K divided among workgroups; against the float64 oracle, within the bound oracle.rows derives for it."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402
from rows_cases import close, cuda, weights  # noqa: E402

FORMATS = [("mxfp4", "mxfp4"), ("mxfp4", "mxfp8"), ("mxfp8", "mxfp8")]


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def _check(dv, w_form, x_form, rows, n, k, gated=False):
    rng = np.random.default_rng(rows + n + k)
    w, x = weights(rng, w_form, n, k), weights(rng, x_form, rows, k)
    if gated:
        w[1][...] += 2  # gates of some size
    lin = dv.Linear(*map(cuda, w), gated=gated)
    assert close(lin(*map(cuda, x)), *oracle.product(*w, *x, gated=gated))
    return lin


# Every number of pairs of 128-wide blocks of K from less than the copies run ahead to more, whole and not.
@pytest.mark.parametrize("k", [128, 256, 384, 512, 640, 768, 1024, 1152, 1408, 1664, 2176])
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_small_tiles_alone(dv, w_form, x_form, k):
    _check(dv, w_form, x_form, 289, 1032, k)


@pytest.mark.parametrize("k", [128, 256, 384, 640, 896, 1280])
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_small_tiles_by_two(dv, w_form, x_form, k):
    _check(dv, w_form, x_form, 1100, 4104, k)


@pytest.mark.parametrize("k", [128, 384, 512, 1152])
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_large_tiles(dv, w_form, x_form, k):
    _check(dv, w_form, x_form, 2060, 4104, k)


def test_large_tiles_gated(dv):
    _check(dv, "mxfp4", "mxfp8", 2060, 4160, 640, gated=True)


@pytest.mark.parametrize("form", ["gather", "scatter"])
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_large_tiles_of_every_height(dv, w_form, x_form, form):
    """Groups of 256 rows and a tail of 1 to 8 blocks of 32, not all whole."""
    groups = [256 + 32 * i + (5 if i % 2 else 32) for i in range(8)]
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    pairs = int(offsets[-1]) + 3
    pairs += pairs % 2
    rng = np.random.default_rng(len(form))
    order = rng.permutation(pairs).astype(np.int32)
    gated = form == "gather"
    n, k = 4416, 640
    w = weights(rng, w_form, len(groups), n, k)
    x = weights(rng, x_form, pairs // 2 if gated else pairs, k)
    gather, scatter = (2, False) if gated else (0, True)
    out = torch.full((pairs, n // 2 if gated else n), 5.0, dtype=torch.bfloat16, device="cuda")
    lin = dv.GroupedLinear(*map(cuda, w), gated=gated)
    lin(*map(cuda, x), cuda(offsets), cuda(order), gather, scatter, out)
    exact, slack, written = oracle.grouped(*w, *x, offsets, order, gather, scatter, gated, pairs)
    assert close(out[cuda(written)], exact[written], slack[written])
    assert (out[cuda(~written)] == 5).all()


DIVIDED = [(130, 520, 8320), (40, 264, 16384), (200, 1088, 16512)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,n,k", DIVIDED)
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_divided_k(dv, w_form, x_form, rows, n, k, gated):
    n = (n + 63) // 64 * 64 if gated else n
    lin = _check(dv, w_form, x_form, rows, n, k, gated)
    kind = dv.mx.MXFP4 if x_form == "mxfp4" else dv.mx.MXFP8
    assert dv.mx.mxrows_workspace_bytes(lin._weight, kind, rows) > 0  # (K is divided here)


def test_divided_k_in_two_graphs_and_on_two_streams(dv):
    """Each call has a workspace of its own: replays of two graphs in turn, calls on two streams at once, and eager work
    between them give the eager results."""
    rng = np.random.default_rng(4)
    rows, n, k = 130, 520, 8320
    lin = dv.Linear(*map(cuda, weights(rng, "mxfp4", n, k)))
    xs = [tuple(map(cuda, weights(rng, "mxfp4", rows, k))) for _ in range(2)]
    want = [lin(*x) for x in xs]
    assert not torch.equal(want[0], want[1])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(lin(*x))
        graphs.append(g)
    for _ in range(3):
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
        lin(*xs[0])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i in (0, 1):
            got[i].append(lin(*xs[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in got[i])
