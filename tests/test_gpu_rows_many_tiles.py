"""More tiles than a row of a grid takes (2^20) on an MI355X, and MXFP8 rows that are to be fast past 4 GiB. Values are 1
and -1, so that sums are whole and every kernel gives the same bits."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_rows_wide import _ones, _product, dv  # noqa: E402, F401


@pytest.mark.parametrize("fast", [False, True])
def test_more_tiles_than_a_row_of_the_grid(dv, fast):  # noqa: F811
    torch.manual_seed(1)
    experts, n, k, rows = 1024, 1 << 17, 128, 9
    w = torch.randint(0, 2, (experts, n, k // 2), dtype=torch.uint8, device="cuda").mul_(0x88).add_(0x22)  # MXFP4, in pairs
    ws = torch.full((experts, n, k // 32), 127, dtype=torch.uint8, device="cuda")
    x, xs = _ones(experts * rows, k)
    offsets = torch.arange(0, experts * rows + 1, rows, dtype=torch.int32, device="cuda")
    y = dv.GroupedLinear(w, ws, fast=fast)(x, xs, offsets)
    for e in (0, 1, 511, 1000, 1023):
        both = (w[e] & 0x80).repeat_interleave(2, -1) | 0x38  # as e4m3
        assert torch.equal(y[e * rows:(e + 1) * rows].double(), _product(x[e * rows:(e + 1) * rows], both))


def test_fast_rows_past_4_gib(dv):  # noqa: F811
    torch.manual_seed(2)
    rows, n, k = (1 << 19) + 1077, 136, 8320
    x, xs = _ones(rows, k)
    assert x.numel() > 1 << 32
    w, ws = _ones(n, k)
    y = dv.Linear(w, ws, fast=True)(x, xs)
    for r0, r1 in ((0, 300), (rows // 2, rows // 2 + 77), (rows - 333, rows)):
        assert torch.equal(y[r0:r1].double(), _product(x[r0:r1], w))


def test_fast_results_past_4_gib(dv):  # noqa: F811
    torch.manual_seed(3)
    rows, n, k = 300_005, 8200, 128
    x, xs = _ones(rows, k)
    w, ws = _ones(n, k)
    y = dv.Linear(w, ws, fast=True)(x, xs)
    assert y.numel() * 2 > 1 << 32
    for r0, r1 in ((0, 64), (rows - 200, rows)):
        assert torch.equal(y[r0:r1].double(), _product(x[r0:r1], w))


@pytest.mark.parametrize("rows", [2, 700])
def test_fast_weights_past_4_gib(dv, rows):  # noqa: F811
    torch.manual_seed(4)
    experts, n, k = 161, 4096, 7168
    w, ws = _ones(experts, n, k)
    assert w.numel() > 1 << 32
    grouped, last = dv.GroupedLinear(w, ws, fast=True), dv.Linear(w[-1].clone(), ws[-1].clone(), fast=True)
    x, xs = _ones(rows, k)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = rows
    assert torch.equal(grouped(x, xs, offsets), last(x, xs))
