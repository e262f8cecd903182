"""mxfp4_quantize and mxfp4_dequantize on an MI355X, bit for bit against the oracle."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def _check(dv, x):
    codes, scales = dv.quantize4(x)
    want, want_s = oracle.quantize4(x.cpu().double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want)
    values = oracle.values(want, want_s)
    for t in TYPES.values():
        got = dv.dequantize4(codes, scales, t)
        with np.errstate(over="ignore"):
            assert torch.equal(got.cpu().nan_to_num(7.0), torch.from_numpy(values).to(t).nan_to_num(7.0))
    return codes, scales


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("rows,k", [(1, 32), (3, 96), (17, 160), (130, 256), (5, 4128)])
def test_random_rows(dv, dtype, rows, k):
    g = torch.Generator().manual_seed(rows * k)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-30, 12, (rows, 1), generator=g).float())
    _check(dv, x.to(TYPES[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("mixed", [False, True])
def test_all_patterns(dv, dtype, mixed):
    bits = np.arange(65536, dtype=np.uint16)
    if mixed:  # neighbours of very different sizes
        bits = np.random.default_rng(2).permutation(bits)
    x = torch.from_numpy(bits.view(np.int16).reshape(16, 4096)).view(TYPES[dtype]).cuda()
    _check(dv, x)


def test_borders_in_float32(dv):
    """The borders of the codes and their neighbours, at scales from the smallest to the largest."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=np.float32)
    around = np.concatenate([borders, np.nextafter(borders, np.float32(0)), np.nextafter(borders[:7], np.float32(9)),
                             [np.float32(6.0)]])
    block = np.concatenate([around[:24], -around[:8]]).astype(np.float32)
    rows = []
    for e in (-127, -126, -60, 0, 60, 125):
        rows.append(np.ldexp(block.astype(np.float64), e).astype(np.float32))
    rows.append(np.full(32, 3.0e38, np.float32))
    rows.append(np.full(32, 1e-45, np.float32))
    _check(dv, torch.from_numpy(np.stack(rows)).cuda())


def test_special_blocks(dv):
    x = torch.randn(4, 128, generator=torch.Generator().manual_seed(1))
    x[0, 5], x[0, 40], x[1, 64] = float("inf"), float("-inf"), float("nan")
    x[2, :32], x[3, 96:] = 0.0, -0.0
    for t in TYPES.values():
        _check(dv, x.to(t).cuda())


def test_row_strides_and_given_outputs(dv):
    g = torch.Generator().manual_seed(4)
    wide = torch.randn(9, 96 + 40, generator=g).bfloat16().cuda()
    x = wide[:, 8:104]
    codes = torch.full((11, 48), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((11, 3), 0xCD, dtype=torch.uint8, device="cuda")
    dv.quantize4(x, codes[1:10], scales[1:10])
    want, want_s = oracle.quantize4(x.cpu().double().numpy())
    assert np.array_equal(codes[1:10].cpu().numpy(), want) and np.array_equal(scales[1:10].cpu().numpy(), want_s)
    for edge in (0, 10):  # the rows beside them are as they were
        assert (codes[edge] == 0xAB).all() and (scales[edge] == 0xCD).all()
    out = torch.empty(9, 96, device="cuda")
    assert dv.dequantize4(codes[1:10], scales[1:10], torch.float32, out) is out
    one = wide[3:4, 8:104]  # one row of any stride
    assert torch.equal(dv.quantize4(one)[0], codes[4:5])


def test_refusals(dv):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    codes, scales = dv.quantize4(x)
    for call in (lambda: dv.quantize4(x.int()), lambda: dv.quantize4(x[:, ::2]), lambda: dv.quantize4(x[:, 1:33]),
                 lambda: dv.quantize4(x[:, :48]), lambda: dv.quantize4(x[0]), lambda: dv.quantize4(x, scales),
                 lambda: dv.quantize4(x, None, codes), lambda: dv.dequantize4(codes, codes),
                 lambda: dv.dequantize4(codes, scales, torch.int32), lambda: dv.dequantize4(x, scales),
                 lambda: dv.dequantize4(codes, scales, torch.float32, x),
                 lambda: dv.quantize4(torch.zeros(4, 67, dtype=torch.bfloat16, device="cuda")[:, :64]),
                 lambda: dv.quantize4(x[:0]), lambda: dv.quantize4(x.requires_grad_())):
        with pytest.raises(ValueError):
            call()
