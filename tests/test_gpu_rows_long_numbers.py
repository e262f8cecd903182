"""Sizes and counts of 2^32 and a little more on an MI355X: refused, where the library's 32 bits would hold the little
alone. Nothing is launched."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from rows_cases import cuda, weights  # noqa: E402

PAST = 1 << 32


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def test_long_rows(dv):
    x = torch.empty(1, PAST + 32, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: dv.quantize4(x), lambda: dv.quantize8(x),
                 lambda: dv.dequantize4(x.view(torch.uint8)[:, : PAST // 2 + 16], x.view(torch.uint8)[:, : PAST // 32 + 1]),
                 lambda: dv.combine(x, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda"),
                                    4)):
        with pytest.raises(ValueError):
            call()


def test_long_rows_of_a_weight(dv):
    w = torch.empty(8, PAST // 2 + 64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        dv.Linear(w, torch.empty(8, PAST // 32 + 4, dtype=torch.uint8, device="cuda"))


def test_many_tokens(dv):
    ids = torch.empty(PAST + 8, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dv.sort_pairs(ids, 4)


@pytest.mark.parametrize("off", [PAST, -PAST])
def test_counts(dv, off):
    rng = np.random.default_rng(1)
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    y = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    lin = dv.GroupedLinear(*map(cuda, weights(rng, "mxfp4", 2, 64, 128)))
    x, xs = map(cuda, weights(rng, "mxfp4", 8, 128))
    order, offsets = dv.sort_pairs(ids, 2)
    lin(x, xs, offsets, order, 2)
    for call in (lambda: dv.sort_pairs(ids, 2 + off), lambda: dv.combine(y, ids, torch.ones(8, 2, device="cuda"), 2 + off),
                 lambda: lin(x, xs, offsets, order, 2 + off)):
        with pytest.raises(ValueError):
            call()
