"""mxmoe_sort and mxmoe_combine on an MI355X against the oracle."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402
from rows_cases import close, cuda  # noqa: E402


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def _sorted(dv, ids, experts):
    order, offsets = dv.sort_pairs(cuda(ids), experts)
    flat = ids.ravel().astype(np.int64)
    key = np.where((flat < 0) | (flat >= experts), experts, flat)
    assert np.array_equal(order.cpu().numpy(), np.argsort(key, kind="stable"))
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(experts + 1)))
    return order, offsets


# One workgroup's chunk is 4096 pairs, a wave's round 64.
@pytest.mark.parametrize("tokens,top_k,experts", [
    (1, 1, 1), (1, 8, 64), (7, 3, 5), (64, 1, 2), (65, 1, 1024), (511, 8, 256), (512, 8, 256), (513, 8, 257),
    (4097, 1, 3), (4096, 2, 1024), (1000, 32, 63), (16384, 8, 256), (70000, 2, 8)])
def test_sort(dv, tokens, top_k, experts):
    rng = np.random.default_rng(tokens * top_k + experts)
    ids = rng.integers(0, experts, (tokens, top_k)).astype(np.int32)
    _sorted(dv, ids, experts)
    ids[rng.random(ids.shape) < 0.3] = -1
    ids[rng.random(ids.shape) < 0.1] = experts
    _sorted(dv, ids, experts)
    _sorted(dv, np.sort(ids.ravel()).reshape(ids.shape), experts)
    _sorted(dv, np.full_like(ids, experts - 1), experts)
    _sorted(dv, np.full_like(ids, -(1 << 31)), experts)


def test_sort_of_many_pairs(dv):
    """More chunks than workgroups: a chunk is longer than 4096."""
    ids = np.random.default_rng(1).integers(-1, 40, (300001, 5)).astype(np.int32)
    _sorted(dv, ids, 39)


def test_sort_matches_the_oracle(dv):
    ids = np.random.default_rng(2).integers(-1, 9, (50, 4)).astype(np.int32)
    order, offsets = dv.sort_pairs(cuda(ids), 8)
    want = oracle.sort_pairs(ids, 8)
    assert np.array_equal(order.cpu().numpy(), want[0]) and np.array_equal(offsets.cpu().numpy(), want[1])


@pytest.mark.parametrize("tokens,top_k,hidden", [(1, 1, 8), (3, 8, 1024), (5, 9, 1032), (2, 32, 2056), (300, 2, 128),
                                                 (70000, 1, 16)])
def test_combine(dv, tokens, top_k, hidden):
    rng = np.random.default_rng(tokens + hidden)
    y = torch.randn(tokens * top_k, hidden, generator=torch.Generator().manual_seed(hidden)).bfloat16()
    ids = rng.integers(-1, 6, (tokens, top_k)).astype(np.int32)
    w = rng.standard_normal((tokens, top_k)).astype(np.float32)
    lost = torch.from_numpy((ids < 0) | (ids >= 5)).flatten()
    y[lost] = float("nan")  # not read
    out = torch.full((tokens + 2, hidden), 5.0, dtype=torch.bfloat16, device="cuda")
    got = dv.combine(y.cuda(), cuda(ids), cuda(w), 5, out[1:-1])
    assert close(got, *oracle.combine(y.double().numpy().reshape(tokens, top_k, hidden), ids, w, 5))
    assert (out[0] == 5).all() and (out[-1] == 5).all()
    assert (got[torch.from_numpy(((ids < 0) | (ids >= 5)).all(1)).cuda()] == 0).all()


def test_combine_keeps_infinities_and_nan_to_their_tokens(dv):
    y = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    y[1, 3], y[2, 5] = float("inf"), float("nan")
    ids = cuda(np.array([[0], [0], [0], [0]], dtype=np.int32))
    got = dv.combine(y, ids, torch.ones(4, 1, device="cuda"), 1)
    assert torch.equal(got.nan_to_num(7.0), y.nan_to_num(7.0))


def test_refusals(dv):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    y = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for call in (lambda: dv.sort_pairs(ids, 0), lambda: dv.sort_pairs(ids, 1025), lambda: dv.sort_pairs(ids.long(), 4),
                 lambda: dv.sort_pairs(ids[0], 4), lambda: dv.sort_pairs(ids, 4, order=ids),
                 lambda: dv.sort_pairs(ids, 4, offsets=ids.flatten()[:4]), lambda: dv.sort_pairs(ids[:0], 4),
                 lambda: dv.sort_pairs(ids.t(), 4), lambda: dv.combine(y[:7], ids, w, 4), lambda: dv.combine(y, ids, ids, 4),
                 lambda: dv.combine(y.float(), ids, w, 4), lambda: dv.combine(y[:, :60].contiguous(), ids, w, 4),
                 lambda: dv.combine(y, ids, w, 0), lambda: dv.combine(y, ids, w, 4, out=y),
                 lambda: dv.combine(y, ids, w.requires_grad_(), 4)):
        with pytest.raises(ValueError):
            call()
