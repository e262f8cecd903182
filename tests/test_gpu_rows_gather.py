"""mxmoe_grouped with orders that lead far into x on an MI355X: entries up to 2^24 rows times 32 choices."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from rows_cases import cuda, weights  # noqa: E402

ROWS = 1 << 24


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


@pytest.mark.parametrize("x_form,fast", [("mxfp4", False), ("mxfp8", False), ("mxfp8", True)])
def test_entries_of_a_long_order(dv, x_form, fast):
    """Before a multiple of the number of choices, in the last rows of x and at the first entries that a product with a
    32-bit reciprocal of 2^32 / choices gets wrong; few rows (streamed) and many (by tiles)."""
    k = 128
    codes = torch.randint(0, 256 if x_form == "mxfp4" else 0x7F, (ROWS, k // 2 if x_form == "mxfp4" else k),
                          dtype=torch.uint8, device="cuda")
    scales = torch.randint(120, 130, (ROWS, k // 32), dtype=torch.uint8, device="cuda")
    lin = dv.GroupedLinear(*map(cuda, weights(np.random.default_rng(1), "mxfp4", 1, 136, k)), fast=fast)
    for gather in range(1, 33):
        first = next((o for j in range(1 << 10) for o in [(1 << 27) + j]
                      if gather > 1 and o // gather < ROWS and (o * ((1 << 32) // gather + 1)) >> 32 != o // gather), gather)
        # From the last row down, and before multiples below the first wrong entry and 2^31's neighbours' quotients.
        entries = [ROWS * gather - 1 - j for j in range(4)] + [first, first - 1, first + 1]
        entries += [m * gather - 1 for m in (1, 2, 1 << 20, (1 << 22) + 1, (1 << 23) + 1, ROWS - 1)]
        for count in (len(entries), 300):
            order = (entries * 30)[:count]
            offsets = cuda(np.array([0, count], dtype=np.int32))
            at = cuda(np.array([o // gather for o in order], dtype=np.int64))
            want = lin(codes[at], scales[at], offsets)
            got = lin(codes, scales, offsets, cuda(np.array(order, dtype=np.int32)), gather)
            assert torch.equal(got.view(torch.int16), want.view(torch.int16)), (gather, count)
