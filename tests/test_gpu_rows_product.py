"""mxrows_product on an MI355X against the float64 oracle, within the bound oracle.rows derives for it."""

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


def _run(dv, w, ws, x, xs, gated=False, **kw):
    return dv.Linear(cuda(w), cuda(ws), gated=gated)(cuda(x), cuda(xs), **kw)


# From one row to more than a tile of any kernel holds, one past its edges; n with a last row block that is not whole; k
# with and without a half of its last pair.
SIZES = [(1, 8, 128), (1, 64, 256), (2, 40, 384), (8, 96, 1024), (31, 200, 640), (32, 256, 2048), (33, 72, 896),
         (64, 320, 512), (65, 264, 1152), (127, 136, 256), (128, 128, 128), (129, 520, 768), (200, 264, 4096),
         (255, 256, 384), (257, 512, 512), (300, 1032, 640), (513, 264, 256), (1025, 136, 384)]


@pytest.mark.parametrize("w_form,x_form", FORMATS)
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_sizes(dv, w_form, x_form, rows, n, k):
    rng = np.random.default_rng(rows * n + k)
    w, x = weights(rng, w_form, n, k), weights(rng, x_form, rows, k)
    assert close(_run(dv, *w, *x), *oracle.product(*w, *x))


@pytest.mark.parametrize("w_form,x_form", FORMATS)
@pytest.mark.parametrize("rows,n,k", [(1, 64, 128), (5, 192, 640), (40, 320, 512), (130, 576, 384), (260, 1088, 256)])
def test_gated(dv, w_form, x_form, rows, n, k):
    rng = np.random.default_rng(rows + n * k)
    w, x = weights(rng, w_form, n, k), weights(rng, x_form, rows, k)
    w[1][...] += 2  # gates of some size
    assert close(_run(dv, *w, *x, gated=True), *oracle.product(*w, *x, gated=True))


def _one_hot(rows, k, code):
    """Row r has one nonzero code, at K position 37 r % k."""
    c = np.zeros((rows, k), dtype=np.uint8)
    c[np.arange(rows), 37 * np.arange(rows) % k] = code
    return c


@pytest.mark.parametrize("rows", [24, 300])
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_every_position(dv, w_form, x_form, rows):
    """One nonzero value in each row of x picks single values of W, with their own scales: exact."""
    n, k = 264, 640
    rng = np.random.default_rng(7)
    w, ws = weights(rng, w_form, n, k)
    ws = rng.integers(100, 150, ws.shape, dtype=np.uint8)
    xs = rng.integers(100, 150, (rows, k // 32), dtype=np.uint8)
    x = _one_hot(rows, k, 3 if x_form == "mxfp4" else 0x3C)  # 1.5
    x = oracle.pack4(x) if x_form == "mxfp4" else x
    exact, _ = oracle.product(w, ws, x, xs)
    assert np.array_equal(f64(_run(dv, w, ws, x, xs)), exact)


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("w_form,x_form", FORMATS)
def test_ends_of_the_scales(dv, w_form, x_form, rows):
    """Scale bytes 0 and 254 in the same row: products from 2^-254 to 2^254; NaN where a scale byte is 255, in its rows and
    columns alone."""
    n, k = 64, 256
    one, two = (2, 4) if w_form == "mxfp4" else (0x38, 0x40)
    xone = 2 if x_form == "mxfp4" else 0x38
    w, x = np.full((n, k), one, dtype=np.uint8), np.full((rows, k), xone, dtype=np.uint8)
    w[1] = two
    w, x = (oracle.pack4(w) if w_form == "mxfp4" else w), (oracle.pack4(x) if x_form == "mxfp4" else x)
    ws, xs = np.full((n, 8), 127, dtype=np.uint8), np.full((rows, 8), 127, dtype=np.uint8)
    ws[2], ws[3], ws[4, 5] = 0, 254, 255
    xs[1], xs[2, 7] = 0, 255
    got = f64(_run(dv, w, ws, x, xs))
    assert np.isnan(got[2]).all() and np.isnan(got[:, 4]).all()
    fine = got[:, np.arange(n) != 4][np.arange(rows) != 2]
    assert not np.isnan(fine).any()
    assert got[0, 0] == k and got[0, 1] == 2 * k and got[0, 2] == k * 2.0**-127 and got[0, 3] == np.inf
    assert got[1, 0] == k * 2.0**-127 and got[1, 2] == 0 and got[1, 3] == k  # 2^-254 is lost


def test_small_products_beside_large_ones(dv):
    """MXFP4 by MXFP4 loses none: 6 * 6 beside 0.5 * 0.5 that others cancel. With MXFP8 what is lost is within the bound."""
    k = 512
    w, x = np.full((8, k), 1, dtype=np.uint8), np.full((2, k), 1, dtype=np.uint8)
    w[:, 0::8], x[:, 0::8] = 7, 7
    w[:, 8::16] |= 8  # every second large product is negative
    ws, xs = np.full((8, k // 32), 127, dtype=np.uint8), np.full((2, k // 32), 127, dtype=np.uint8)
    got = _run(dv, oracle.pack4(w), ws, oracle.pack4(x), xs)
    assert (f64(got) == 7 * 64 * 0.25).all()
    x8 = np.full((2, k), 0x01, dtype=np.uint8)  # 2^-9
    x8[:, 0::8] = 0x7E                          # 448
    pair = oracle.pack4(w), ws, x8, xs
    assert close(_run(dv, *pair), *oracle.product(*pair))


def test_bf16_rows_are_quantized(dv):
    rng = np.random.default_rng(9)
    w, ws = weights(rng, "mxfp4", 96, 384)
    x = torch.randn(37, 384, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    for activation, quantize in (("mxfp4", dv.quantize4), ("mxfp8", dv.quantize8)):
        lin = dv.Linear(cuda(w), cuda(ws), activation=activation)
        assert torch.equal(lin(x), lin(*quantize(x)))
    assert dv.Linear(cuda(w), cuda(ws)).activation == 4


def test_a_given_output_and_the_rows_beside_it(dv):
    rng = np.random.default_rng(10)
    for rows in (5, 70, 300):
        w, x = weights(rng, "mxfp4", 72, 256), weights(rng, "mxfp4", rows, 256)
        lin = dv.Linear(*map(cuda, w))
        out = torch.full((rows + 2, 72), 3.0, dtype=torch.bfloat16, device="cuda")
        assert lin(*map(cuda, x), out=out[1:-1]).data_ptr() == out[1:].data_ptr()
        assert torch.equal(out[1:-1], lin(*map(cuda, x)))
        assert (out[0] == 3).all() and (out[-1] == 3).all()


def test_the_same_bits_on_every_call_and_for_every_batch(dv):
    rng = np.random.default_rng(11)
    w, x = weights(rng, "mxfp4", 256, 2048), weights(rng, "mxfp4", 300, 2048)
    lin = dv.Linear(*map(cuda, w))
    x, xs = map(cuda, x)
    whole = lin(x, xs)
    for _ in range(3):
        assert torch.equal(lin(x, xs), whole)


def test_refusals(dv):
    rng = np.random.default_rng(12)
    w, ws = map(cuda, weights(rng, "mxfp4", 64, 256))
    w8, ws8 = map(cuda, weights(rng, "mxfp8", 64, 256))
    x, xs = map(cuda, weights(rng, "mxfp4", 4, 256))
    lin, lin8 = dv.Linear(w, ws), dv.Linear(w8, ws8)
    bf = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: dv.Linear(w, ws[:, :4]), lambda: dv.Linear(w[:, :100], ws), lambda: dv.Linear(w[:60], ws[:60]),
                 lambda: dv.Linear(w[:32], ws[:32], gated=True), lambda: dv.Linear(w.unsqueeze(0), ws.unsqueeze(0)),
                 lambda: dv.Linear(w, ws, activation="bf16"), lambda: dv.Linear(w8, ws8, activation="mxfp4"),
                 lambda: dv.Linear(w, None), lambda: lin8(x, xs), lambda: lin(x, xs[:3]), lambda: lin(x[:, :64], xs),
                 lambda: lin(x, None), lambda: lin(bf, xs), lambda: lin(bf[:, :128]), lambda: lin(x[:0], xs[:0]),
                 lambda: lin(x, xs, out=bf), lambda: lin(x[0], xs[0]), lambda: lin(bf.requires_grad_())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(AttributeError):
        lin.w = w
