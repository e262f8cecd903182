"""Gates far below zero beside large ups on an MI355X: silu(gate) is below FP32's normal range from -91 on, its product with
up is not. Sums of one product each, so that gate and up are exact."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402
from rows_cases import cuda, f64  # noqa: E402


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


# A stream, a tile of 128 alone, K divided.
@pytest.mark.parametrize("rows,k", [(3, 128), (300, 128), (130, 8320)])
@pytest.mark.parametrize("x_form", ["mxfp4", "mxfp8"])
def test_gates_below_the_normal_range(dv, rows, k, x_form):
    """Within the bound of silu and its product (oracle.rows) and a BF16 step."""
    rng = np.random.default_rng(rows)
    half = 256
    w = np.zeros((2 * half, k), dtype=np.uint8)
    ws = np.full((2 * half, k // 32), 127, dtype=np.uint8)
    w[:half, 0] = 8 | rng.integers(2, 8, half)                    # -1 to -6
    ws[:half, 0] = 127 + rng.integers(3, 6, half)                 # by 8, 16 or 32
    w[half:, 0] = rng.integers(2, 8, half) | 8 * rng.integers(0, 2, half)
    ws[half:, 0] = 127 + rng.choice([0, 60, 100, 120, 125], half)
    w[:8, 0], ws[:8, 0] = [2, 7, 10, 15, 1, 9, 0, 8], 127         # and gates of both signs near zero
    x = np.zeros((rows, k), dtype=np.uint8)
    x[:, 0] = 2 if x_form == "mxfp4" else 0x38                    # 1
    xs = np.full((rows, k // 32), 127, dtype=np.uint8)
    g, u = np.split(oracle.values(oracle.pack4(w), ws)[:, 0], 2)
    want = g / (1 + np.exp(-g)) * u
    lin = dv.Linear(cuda(oracle.pack4(w)), cuda(ws), gated=True)
    got = f64(lin(cuda(oracle.pack4(x) if x_form == "mxfp4" else x), cuda(xs)))
    assert (g < -100).sum() > 10 and (np.abs(want[g < -100]) > 2.0**-100).any()
    bound = oracle.bf16_bound(want, oracle.GATE_ROUNDING * (10 + np.abs(g)) * np.abs(want))
    past = np.abs(want) > 2.0**128 * (1 - 2.0**-9)  # (a gate of 6 by the largest ups: infinite in BF16)
    assert np.array_equal(got[:, past], np.broadcast_to(np.copysign(np.inf, want[past]), got[:, past].shape))
    assert (np.abs(got - want) <= bound)[:, ~past].all()
