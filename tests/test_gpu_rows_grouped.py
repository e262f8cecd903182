"""mxmoe_grouped on an MI355X against the float64 oracle: ragged groups, experts without rows, gathered and scattered
rows."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402
from rows_cases import close, cuda, f64, weights  # noqa: E402

FORMATS = [("mxfp4", "mxfp4"), ("mxfp4", "mxfp8"), ("mxfp8", "mxfp8")]


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


GROUPS = {
    "one row": [0, 0, 1, 0],
    "few": [3, 0, 1, 2, 0, 5],
    "edges": [32, 1, 31, 33, 0, 64],
    "ragged": [0, 129, 7, 0, 256, 60, 1, 0],
    "all in one": [0, 0, 300],
    "many experts": [(i * 7) % 5 for i in range(130)],
    "large": [513, 255, 0, 300],
}


def _layout(groups, top_k, rng):
    """offsets, and an order of pairs whose tokens are distinct per expert as far as that can be; two rows more than the
    groups have, without an expert."""
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    rows = -(-(int(offsets[-1]) + 2) // top_k) * top_k
    return offsets, rng.permutation(rows).astype(np.int32), rows


@pytest.mark.parametrize("w_form,x_form", FORMATS)
@pytest.mark.parametrize("form", ["gather", "scatter", "both", "plain"])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_groups(dv, name, form, w_form, x_form):
    groups = GROUPS[name]
    rng = np.random.default_rng(len(name) + len(form))
    gated = form in ("gather", "both")
    n, k, top_k = (192 if gated else 72), 384, 3
    offsets, order, rows = _layout(groups, top_k, rng)
    w = weights(rng, w_form, len(groups), n, k)
    gather = top_k if form in ("gather", "both") else 0
    x = weights(rng, x_form, rows // top_k if gather else rows, k)
    scatter = form in ("scatter", "both")
    out = torch.full((rows, n // 2 if gated else n), 5.0, dtype=torch.bfloat16, device="cuda")
    lin = dv.GroupedLinear(*map(cuda, w), gated=gated)
    got = lin(*map(cuda, x), cuda(offsets), None if form == "plain" else cuda(order), gather, scatter, out)
    exact, slack, written = oracle.grouped(*w, *x, offsets, order, gather, scatter, gated, rows)
    assert got is out and close(got[cuda(written)], exact[written], slack[written])
    assert (f64(got)[~written] == 5).all()  # rows without an expert are as they were


def test_one_expert_is_the_product(dv):
    rng = np.random.default_rng(1)
    w, x = weights(rng, "mxfp4", 1, 136, 640), weights(rng, "mxfp4", 150, 640)
    one = dv.Linear(cuda(w[0][0]), cuda(w[1][0]))(*map(cuda, x))
    lin = dv.GroupedLinear(*map(cuda, w))
    assert torch.equal(lin(*map(cuda, x), cuda(np.array([0, 150], dtype=np.int32))), one)


def test_values_that_lead_nowhere(dv):
    """Entries of order outside x and out, and offsets outside the rows, reach no other memory; the others' results stand."""
    rng = np.random.default_rng(2)
    w, x = weights(rng, "mxfp4", 3, 64, 256), weights(rng, "mxfp4", 20, 256)
    lin = dv.GroupedLinear(*map(cuda, w))
    order = np.arange(40, dtype=np.int32)
    offsets = np.array([0, 10, 30, 40], dtype=np.int32)
    want = lin(*map(cuda, x), cuda(offsets), cuda(order), 2)
    bad = order.copy()
    bad[[0, 15, 39]] = [-1, 1 << 30, -(1 << 31)]
    got = lin(*map(cuda, x), cuda(offsets), cuda(bad), 2)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[0, 15, 39]] = False
    assert torch.equal(got[keep], want[keep])
    out = torch.full((42, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lin(*map(cuda, x), cuda(offsets), cuda(bad), 2, True, out[1:41])
    assert torch.equal(out[1:41][keep], want[keep])
    assert (out[[0, 1, 16, 40, 41]] == 5).all()
    wide = cuda(np.array([-5, 10, 30, 1000], dtype=np.int32))
    assert torch.equal(lin(*map(cuda, x), wide, cuda(order), 2), want)


def test_bf16_rows_and_refusals(dv):
    rng = np.random.default_rng(3)
    w, ws = map(cuda, weights(rng, "mxfp4", 3, 64, 256))
    x, xs = map(cuda, weights(rng, "mxfp4", 6, 256))
    offsets = cuda(np.array([0, 2, 2, 6], dtype=np.int32))
    order = cuda(np.arange(6, dtype=np.int32))
    lin = dv.GroupedLinear(w, ws)
    bf = torch.randn(6, 256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    assert torch.equal(lin(bf, None, offsets), lin(*dv.quantize4(bf), offsets))
    for call in (lambda: lin(x, xs, offsets[:3]), lambda: lin(x, xs, offsets.long()), lambda: lin(x, xs, None),
                 lambda: lin(x, xs, offsets, None, 2), lambda: lin(x, xs, offsets, None, 0, True),
                 lambda: lin(x, xs, offsets, order[:4]), lambda: lin(x, xs, offsets, order.float()),
                 lambda: lin(x, xs, offsets, order, -1), lambda: lin(x, xs, offsets, [0, 1]),
                 lambda: lin(x, xs, offsets, out=bf), lambda: dv.GroupedLinear(w[0], ws[0]),
                 lambda: lin(bf.requires_grad_(), None, offsets)):
        with pytest.raises(ValueError):
            call()
