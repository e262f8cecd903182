"""Products of any number of rows past 4 GiB of x, of results and of weights on an MI355X: the rows and the expert that lie
behind the border against a call on them alone. Values are 1 and -1, so that sums are whole and every order gives the same
bits."""

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


def _ones(*shape):
    """e4m3 codes of 1 and -1, and their scale bytes."""
    codes = torch.randint(0, 2, shape, dtype=torch.uint8, device="cuda").mul_(0x80).add_(0x38)
    return codes, torch.full((*shape[:-1], shape[-1] // 32), 127, dtype=torch.uint8, device="cuda")


def _product(x, w):
    value = lambda c: 1.0 - (c >> 7).double() * 2  # noqa: E731
    return (value(x) @ value(w).T).bfloat16().double()


def test_rows_past_4_gib(dv):
    torch.manual_seed(1)
    rows, n, k = (1 << 19) + 1077, 136, 8320
    x, xs = _ones(rows, k)
    assert x.numel() > 1 << 32
    w, ws = _ones(n, k)
    y = dv.Linear(w, ws)(x, xs)
    for r0, r1 in ((0, 300), (rows // 2, rows // 2 + 77), (rows - 333, rows)):
        assert torch.equal(y[r0:r1].double(), _product(x[r0:r1], w))


def test_results_past_4_gib(dv):
    torch.manual_seed(2)
    rows, n, k = 300_005, 8200, 128
    x, xs = _ones(rows, k)
    w, ws = _ones(n, k)
    y = dv.Linear(w, ws)(x, xs)
    assert y.numel() * 2 > 1 << 32
    for r0, r1 in ((0, 64), (rows - 200, rows)):
        assert torch.equal(y[r0:r1].double(), _product(x[r0:r1], w))


@pytest.mark.parametrize("rows", [2, 700])
def test_weights_past_4_gib(dv, rows):
    torch.manual_seed(3)
    experts, n, k = 161, 4096, 7168
    w, ws = _ones(experts, n, k)
    assert w.numel() > 1 << 32
    grouped, last = dv.GroupedLinear(w, ws), dv.Linear(w[-1].clone(), ws[-1].clone())
    x, xs = _ones(rows, k)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = rows
    assert torch.equal(grouped(x, xs, offsets), last(x, xs))
