"""Products of MXFP8 rows that are to be fast (MXG_MXFP8_FAST) on an MI355X, by each of their kernels, against the float64
oracle within the bound that oracle.rows derives for the scaled instruction."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402
from rows_cases import close, cuda, weights  # noqa: E402

W_FORMS = ["mxfp4", "mxfp8"]


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


# Streams, K divided, tiles of 128 alone on a CU and by two, tiles of 256.
SIZES = [(1, 40, 128), (8, 96, 1024), (33, 136, 4096), (130, 520, 8320), (40, 264, 16384), (200, 1088, 16512),
         *((289, 1032, k) for k in (128, 256, 384, 512, 640, 768, 1024, 1152, 1408, 1664, 2176)),
         *((1100, 4104, k) for k in (128, 256, 384, 640, 896, 1280)), *((2060, 4104, k) for k in (128, 384, 512, 1152))]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("w_form", W_FORMS)
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_sizes(dv, w_form, rows, n, k, gated):
    rng = np.random.default_rng(rows * n + k)
    n = (n + 63) // 64 * 64 if gated else n
    w, x = weights(rng, w_form, n, k), weights(rng, "mxfp8", rows, k)
    if gated:
        w[1][...] += 2  # gates of some size
    lin = dv.Linear(*map(cuda, w), gated=gated, fast=True)
    assert close(lin(*map(cuda, x)), *oracle.product(*w, *x, gated=gated, fast=True))


@pytest.mark.parametrize("groups", [[3, 0, 1, 2, 0, 5], [0, 129, 7, 0, 256, 60, 1, 0],
                                    [256 + 32 * i + (5 if i % 2 else 32) for i in range(8)]])
@pytest.mark.parametrize("w_form", W_FORMS)
def test_experts(dv, w_form, groups):
    rng = np.random.default_rng(len(groups))
    offsets = np.concatenate([[0], np.cumsum(groups)]).astype(np.int32)
    rows = int(offsets[-1]) + int(offsets[-1]) % 2
    order = rng.permutation(rows).astype(np.int32)
    n, k = (4416, 640) if rows > 2000 else (192, 2304)
    w = weights(rng, w_form, len(groups), n, k)
    for gather, scatter in ((2, False), (0, True)):
        x = weights(rng, "mxfp8", rows // 2 if gather else rows, k)
        out = torch.full((rows, n // 2 if gather else n), 5.0, dtype=torch.bfloat16, device="cuda")
        dv.GroupedLinear(*map(cuda, w), gated=bool(gather), fast=True)(*map(cuda, x), cuda(offsets), cuda(order), gather,
                                                                       scatter, out)
        exact, slack, written = oracle.grouped(*w, *x, offsets, order, gather, scatter, bool(gather), rows, fast=True)
        assert close(out[cuda(written)], exact[written], slack[written])
        assert (out[cuda(~written)] == 5).all()


def test_it_is_a_choice(dv):
    """Small products beside large ones that cancel: lost where the rows are to be fast, kept otherwise; BF16 rows that are
    quantized to MXFP8 and a layer of experts go by the same choice, MXFP4 rows have none to make."""
    from test_gpu_rows_sums import _cancelling, _rounded

    rng = np.random.default_rng(3)
    (w, ws), (x, xs) = _cancelling(rng, "mxfp4", 70, 256, 512)
    exact, slack = oracle.product(w[0], ws[0], x, xs, fast=True)
    args, rows = (cuda(w[0]), cuda(ws[0])), (cuda(x), cuda(xs))
    fast, full = dv.Linear(*args, fast=True), dv.Linear(*args)
    assert torch.equal(full(*rows), _rounded(exact)) and not torch.equal(fast(*rows), _rounded(exact))
    assert close(fast(*rows), exact, slack)
    bf = torch.randn(70, 512, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    fast8 = dv.Linear(*args, activation="mxfp8", fast=True)
    assert torch.equal(fast8(bf), fast(*dv.quantize8(bf)))
    assert torch.equal(fast(bf), full(bf))  # (quantized to MXFP4)
    w2 = _cancelling(rng, "mxfp4", 1, 512, 128)[0]
    layer = dv.PromptExperts(*map(cuda, (w, ws, *w2)), activation="mxfp8", fast=True)
    assert layer.up._mxfp8 == layer.down._mxfp8 == dv.mx.MXFP8_FAST
