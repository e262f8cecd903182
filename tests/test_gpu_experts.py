"""mxmoe_experts on an MI355X against the float64 oracle, within the bound
oracle.decode derives for it."""

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


def _quantized(rng, *shape):
    from workloads import generate

    v = rng.standard_normal((int(np.prod(shape[:-1])), shape[-1])) * shape[-1] ** -0.5
    q, s = generate.quantize_mxfp8(v)
    return q.reshape(shape), s.reshape(*shape[:-1], shape[-1] // 32)


def _bits(values):
    from workloads import generate

    return generate.bf16_bits(np.asarray(values, dtype=np.float32))


def _f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Layer:
    def __init__(self, dv, seed, experts, hidden, inter, pairs=1024):
        rng = np.random.default_rng(seed)
        self.dims = experts, hidden, inter
        self.host = (*_quantized(rng, experts, 2 * inter, hidden),
                     *_quantized(rng, experts, hidden, inter))
        self.layer = dv.Experts(*(torch.from_numpy(v).cuda() for v in self.host), pairs)

    def inputs(self, seed, tokens, top_k):
        rng = np.random.default_rng(seed)
        experts, hidden, _ = self.dims
        x = _bits(rng.standard_normal((tokens, hidden)))
        ids = np.stack([rng.choice(experts, top_k, replace=False) for _ in range(tokens)])
        w = rng.random((tokens, top_k)).astype(np.float32)
        return x, ids.astype(np.int32), w

    def run(self, x, ids, w, **kw):
        t = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
        out = self.layer(t, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), **kw)
        return out

    def check(self, x, ids, w, out=None):
        from oracle import decode

        print(f"experts {self.dims} ids {ids.shape}", flush=True)
        out = self.run(x, ids, w) if out is None else out
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        exact, bound = decode.experts(_f64(x), ids, w, *self.host)
        off = np.abs(got - exact) / bound
        assert np.isfinite(got).all() and off.max() <= 1.0, off.max()
        return got


@pytest.mark.parametrize("tokens,top_k,experts,hidden,inter", [
    (1, 1, 1, 128, 128),      # one K block: seven of eight waves add zeros
    (1, 2, 4, 128, 256), (1, 8, 16, 1024, 512), (2, 3, 5, 384, 896), (3, 2, 8, 896, 384),
    (8, 8, 32, 512, 256), (8, 1, 3, 256, 1152), (7, 4, 4, 640, 128), (5, 2, 64, 1152, 128),
    (17, 2, 4, 256, 128),     # more rows per expert than one chunk holds
    (64, 4, 8, 384, 256), (128, 8, 16, 256, 128), (1024, 1, 2, 128, 128), (1, 64, 64, 128, 128),
])
def test_experts(dv, tokens, top_k, experts, hidden, inter):
    layer = Layer(dv, 31 + tokens, experts, hidden, inter)
    layer.check(*layer.inputs(tokens * 7 + top_k, tokens, top_k))


@pytest.mark.parametrize("tokens,top_k,experts,hidden,inter", [
    (1, 1024, 3, 128, 128), (1024, 1, 1024, 128, 128), (2, 3, 2, 32768, 128),
    (2, 3, 2, 128, 32768), (40, 2, 3, 128, 32768), (40, 2, 3, 32768, 128),
])
def test_ends_of_the_ranges(dv, tokens, top_k, experts, hidden, inter):
    layer = Layer(dv, 3 + tokens, experts, hidden, inter)
    x, ids, w = layer.inputs(tokens + top_k, tokens, min(top_k, experts))
    reps = -(-top_k // experts)  # more choices than experts: each one again
    layer.check(x, np.tile(ids, (1, reps))[:, :top_k].copy(),
                np.tile(w, (1, reps))[:, :top_k].copy())


def test_large_widths(dv):
    layer = Layer(dv, 5, 3, 7168, 2048, 16)
    layer.check(*layer.inputs(6, 4, 2))


def test_ids_outside_and_twice(dv):
    """Ids outside the range add nothing (whole rows and single choices); a row
    may name an expert twice; one expert may take every pair."""
    layer = Layer(dv, 9, 6, 256, 256)
    x, ids, w = layer.inputs(1, 9, 4)
    ids[0] = -1
    ids[1, 2:] = [6, 2**31 - 1]
    ids[2] = 3
    ids[3] = [-(2**31), 1, 1, -1]
    got = layer.check(x, ids, w)
    assert (got[0] == 0).all()
    layer.check(x, np.full_like(ids, 5), w)
    none = layer.run(x, np.full_like(ids, -1), w)
    assert (none == 0).all()


def test_special_values_stay_in_their_row(dv):
    """An infinity or NaN in one row leaves the other rows' bits alone, also
    those that share its expert; a zero weight on a finite row adds nothing."""
    layer = Layer(dv, 10, 4, 256, 128)
    x, ids, w = layer.inputs(2, 6, 2)
    ids[:] = [1, 2]
    clean = layer.run(x, ids, w).clone()
    bad = x.copy()
    bad[3, 5], bad[4, 7] = 0x7F80, 0x7FC0
    got = layer.run(bad, ids, w)
    rest = [0, 1, 2, 5]
    assert torch.equal(got[rest], clean[rest])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[3]).all()
    w[:, 1] = 0
    layer.check(x, ids, w)


def test_zero_codes_and_scales(dv):
    """Experts of zero weights, negative zeros, and scale bytes at both ends of
    the exact range."""
    layer = Layer(dv, 12, 3, 256, 128)
    w13, s13, w2, s2 = layer.host
    w13[0] = 0x80
    w2[1] = 0
    s13[2] = 3
    s2[2] = 246
    layer.layer = dv.Experts(*(torch.from_numpy(v).cuda() for v in layer.host))
    x, ids, w = layer.inputs(4, 5, 2)
    ids[:] = [0, 1]
    assert (layer.check(x, ids, w) == 0).all()
    ids[:] = [2, 0]
    # gate and up are of order 2^-120: their product underflows FP32, as in the oracle's bound
    got = layer.run(x, ids, w)
    assert torch.isfinite(got).all()


def test_outputs_and_rows_behind(dv):
    """Results into a given output; rows behind the last one stay."""
    layer = Layer(dv, 13, 8, 384, 128)
    x, ids, w = layer.inputs(8, 5, 2)
    want = layer.run(x, ids, w)
    out = torch.full((7, 384), 3.0, dtype=torch.bfloat16, device="cuda")
    layer.run(x, ids, w, out=out[1:6])
    assert torch.equal(out[1:6], want) and (out[[0, 6]] == 3).all()


def test_same_bits_every_time(dv):
    """Every workgroup sorts the pairs for itself: experts of several chunks come
    out the same on every call. Another stream, and a workspace holding other
    values."""
    layer = Layer(dv, 14, 4, 512, 384)
    x, ids, w = layer.inputs(3, 40, 2)
    want = layer.run(x, ids, w).clone()
    side = torch.cuda.Stream()
    for i in range(4):
        layer.layer.workspace.fill_(0xFF if i % 2 else 0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = layer.run(x, ids, w)
        side.synchronize()
        assert torch.equal(got, want)


def test_refusals(dv):
    layer = Layer(dv, 15, 4, 256, 128, 8)
    x, ids, w = (torch.from_numpy(v).cuda() for v in layer.inputs(1, 4, 2))
    x = x.view(torch.int16).view(torch.bfloat16)
    for bad in ((x.float(), ids, w), (x[:3], ids, w), (x, ids.long(), w), (x, ids, w.double()),
                (x[:, :128], ids, w), (x.repeat(2, 1), ids.repeat(2, 1), w.repeat(2, 1)),
                (x.cpu(), ids, w), (x, ids[:0], w[:0])):
        with pytest.raises(ValueError):
            layer.layer(*bad)
    with pytest.raises(ValueError):
        dv.Experts(*(torch.from_numpy(v).cuda() for v in layer.host), 1025)


@pytest.mark.parametrize("tokens,top_k,experts,hidden,inter", [
    (40, 1, 1, 256, 384), (33, 2, 2, 1152, 1024), (65, 1, 3, 128, 2048), (9, 8, 8, 512, 128),
    (256, 4, 1000, 128, 128), (24, 3, 3, 2048, 1152), (512, 2, 16, 128, 256),
])
def test_many_rows(dv, tokens, top_k, experts, hidden, inter):
    """Rows copied into column tiles: chunks that end inside a tile, experts of
    one row among full ones, both halves of the pairs."""
    layer = Layer(dv, 77 + tokens, experts, hidden, inter)
    x, ids, w = layer.inputs(tokens + experts, tokens, top_k)
    layer.check(x, ids, w)
    ids[::3, 0] = 0  # one crowded expert, twice in some rows
    ids[1] = -1
    got = layer.check(x, ids, w)
    assert (got[1] == 0).all()
    none = layer.run(x, np.full_like(ids, experts), w)
    assert (none == 0).all()


def test_one_row_set_through_both_paths(dv):
    """A row's result does not depend on the rows beside it: the first 8 of 64
    rows, alone (gathered) and among the others (in column tiles)."""
    layer = Layer(dv, 78, 6, 640, 384)
    x, ids, w = layer.inputs(5, 64, 2)
    many = layer.run(x, ids, w).clone()
    assert torch.equal(layer.run(x[:8].copy(), ids[:8].copy(), w[:8].copy()), many[:8])


def test_captured(dv):
    """Replays of both paths with new inputs, eager calls between."""
    for tokens in (3, 48):
        layer = Layer(dv, 79, 5, 512, 256, 96)
        other = Layer(dv, 79, 5, 512, 256, 96)
        ins = [layer.inputs(s, tokens, 2) for s in range(5)]
        x = torch.empty(tokens, 512, dtype=torch.bfloat16, device="cuda")
        ids = torch.zeros(tokens, 2, dtype=torch.int32, device="cuda")
        w = torch.zeros(tokens, 2, device="cuda")
        out = torch.empty_like(x)
        layer.layer(x.zero_(), ids, w, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.layer(x, ids, w, out=out)
        for bits, i, wt in ins:
            x.copy_(torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16))
            ids.copy_(torch.from_numpy(i))
            w.copy_(torch.from_numpy(wt))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, other.run(bits, i, wt))


def test_pack_is_the_projections_layout(dv):
    """Every expert's packed weight is mxgemm_pack_weight's of its matrix."""
    rng = np.random.default_rng(3)
    q, s = _quantized(rng, 5, 48, 384)
    w, ws = dv.pack_experts(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    one = [dv.pack_weight(torch.from_numpy(q[e]).cuda(), torch.from_numpy(s[e]).cuda(), 48, 384)
           for e in range(5)]
    assert torch.equal(w, torch.cat([a for a, _ in one]))
    for e, (_, b) in enumerate(one):  # (the bytes that round the range words up are not written)
        used = 48 * 12 + 12
        assert torch.equal(ws.view(5, -1)[e, :used], b[:used])
