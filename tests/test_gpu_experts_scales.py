"""mxmoe_experts with scale bytes outside 3..246, where a weight is the BF16
value nearest to its code times its scale: against the float64 oracle, which rounds
the weights so, within the bound it derives."""

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


def _layer(dv, seed, s13, s2, top_code):
    """Scale bytes drawn from s13 and s2; w2's codes below top_code."""
    from test_gpu_experts import Layer

    layer = Layer(dv, seed, 3, 256, 128, 64)
    rng = np.random.default_rng(seed)
    w13, sc13, w2, sc2 = layer.host
    sc13[...] = rng.choice(s13, sc13.shape).astype(np.uint8)
    sc2[...] = rng.choice(s2, sc2.shape).astype(np.uint8)
    w2[...] = (rng.integers(0, top_code, w2.shape) | (rng.integers(0, 2, w2.shape) << 7))
    layer.layer = dv.Experts(*(torch.from_numpy(v).cuda() for v in layer.host), 64)
    return layer


# (w13's bytes, w2's bytes, w2's largest code, the exponent of x): h is the product of
# two sums of w13 x, of order 2^-60 or 2^60, and the results stay inside FP32.
CASES = [
    ([0, 1, 2, 3, 4], [190, 191], 0x7F, 90),
    ([0, 2], [247, 248], 0x48, 90),
    ([130, 131], [0, 1, 2, 3], 0x7F, 24),
    ([150, 151], [0], 0x7F, 24),
    ([110, 111], [247, 250, 254], 0x30, -16),
    ([247, 248, 250], [100, 101], 0x7F, -110),
]


@pytest.mark.parametrize("s13,s2,top,e", CASES)
@pytest.mark.parametrize("tokens", [4, 30])
def test_scales_outside_the_exact_range(dv, s13, s2, top, e, tokens):
    layer = _layer(dv, 40 + e + 200, s13, s2, top)
    if max(s13) > 246:  # codes whose product with the scale is a finite BF16 value
        layer.host[0][...] = (layer.host[0] & 0x80) | (layer.host[0] % 0x40)
        layer.layer = dv.Experts(*(torch.from_numpy(v).cuda() for v in layer.host), 64)
    x, ids, w = layer.inputs(7, tokens, 2)
    x = ((x & 0x8000) | ((((x >> 7) & 0xFF).astype(np.int32) + e).clip(1, 254) << 7).astype(
        np.uint16) | (x & 0x7F)).astype(np.uint16)
    with np.errstate(over="ignore"):  # (the oracle's exp of a large negative gate)
        got = layer.check(x, ids, w)
    assert (np.abs(got) > 0).mean() > 0.5
