"""mxgemm_lora on an MI355X against the float64 oracle, within the bound
oracle.decode derives for it, and against mxgemm / mxgemm_publish bit for bit
where no row has an adapter."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import binding, device

    torch.cuda.set_device(0)
    return binding, device


def _f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Case:
    """One projection with `adapters` adapters and inputs of m rows, from a seed."""

    def __init__(self, dv, m, n, k, split_k, rank, adapters, seed=0, dist="normal"):
        from oracle import gemm, quant
        from workloads import generate

        print(f"adapted m={m} n={n} k={k} split_k={split_k} rank={rank}", flush=True)
        rng = np.random.default_rng(seed + 17)
        self.p = p = generate.random_problem(seed + 100 + m + n + k, m, n, k, split_k, dist)
        self.a = generate.bf16_bits((rng.standard_normal((adapters, rank, k)) * k**-0.5)
                                    .astype(np.float32))
        self.b = generate.bf16_bits((8 * rng.standard_normal((adapters, n, rank)))
                                    .astype(np.float32))
        self.scale = rng.uniform(-2, 2, adapters).astype(np.float32)
        self.xb = generate.bf16_activation(seed + 5, m, k, "outliers" if dist == "outliers"
                                           else "normal")
        codes, scales = quant.quantize_bf16(self.xb) if k <= 2048 else generate.quantize_mxfp8(
            _f64(self.xb))
        self.xq = gemm.dequantize(codes, scales)
        self.lin = dv.AdaptedLinear(
            torch.from_numpy(p.w).cuda(), torch.from_numpy(p.ws).cuda(),
            self._bf(self.a), self._bf(self.b), torch.from_numpy(self.scale).cuda(), split_k)
        self.rng = rng

    @staticmethod
    def _bf(bits):
        return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)

    def forms(self):
        from oracle import gemm

        yield (self._bf(self.xb), None), self.xq, _f64(self.xb)
        v = gemm.dequantize(self.p.x, self.p.xs)
        yield (torch.from_numpy(self.p.x).cuda(), torch.from_numpy(self.p.xs).cuda()), v, v

    def check(self, ids):
        from oracle import decode

        ids = np.asarray(ids, dtype=np.int32)
        dev_ids = torch.from_numpy(ids).cuda()
        for (x, xs), shared, own in self.forms():
            out = self.lin(x, dev_ids, x_scale=xs)
            torch.cuda.synchronize()
            got = out.double().cpu().numpy()
            exact, bound = decode.adapted(shared, own, self.p.w, self.p.ws, _f64(self.a),
                                          _f64(self.b), self.scale.astype(np.float64), ids)
            off = np.abs(got - exact) / bound
            assert np.isfinite(got).all() and off.max() <= 1.0, (xs is None, off.max())


@pytest.mark.parametrize("m,n,k,split_k,rank,adapters", [
    (1, 8, 128, 1, 8, 1), (1, 256, 512, 1, 8, 3), (2, 24, 256, 2, 16, 2), (3, 1000, 512, 1, 24, 4),
    (8, 1000, 1024, 2, 128, 5), (8, 520, 2048, 4, 32, 9), (5, 2056, 1024, 8, 64, 3),
    (4, 7168, 2048, 1, 64, 2), (7, 904, 1920, 1, 40, 4), (8, 64, 16384, 8, 16, 2),
    (6, 136, 6400, 1, 120, 6), (8, 4096, 4096, 4, 8, 8),
    # few workgroups, many dot products: others help
    (8, 8, 16384, 1, 128, 3), (8, 64, 4096, 8, 128, 8), (7, 2048, 1024, 1, 128, 2),
    (8, 1024, 2176, 1, 72, 5),
    # more workgroups than a split-K grid may have
    (3, 40960, 512, 1, 16, 4), (8, 33000, 128, 1, 128, 8),
])
def test_adapted(env, m, n, k, split_k, rank, adapters):
    c = Case(env[1], m, n, k, split_k, rank, adapters)
    c.check(c.rng.integers(0, adapters, m))


def test_headline_width(env):
    """N=7168, K=8192, 8 rows, split-K 4, outlier channels, an adapter each."""
    c = Case(env[1], 8, 7168, 8192, 4, 16, 8, dist="outliers")
    c.check([3, 0, 7, 1, 2, 6, 5, 4])


@pytest.mark.parametrize("split_k", [1, 4])
def test_rows_without_adapter(env, split_k):
    """Ids outside the range add nothing: those rows keep mxgemm's bits."""
    mx, dv = env
    c = Case(dv, 8, 1032, 1024, split_k, 16, 3, seed=3)
    c.check([0, -1, 2, 3, 2**31 - 1, 1, -(2**31), 1])
    codes, scales = torch.from_numpy(c.p.x).cuda(), torch.from_numpy(c.p.xs).cuda()
    plain = torch.empty(8, 1032, dtype=torch.bfloat16, device="cuda")
    ws = c.lin.workspace
    mx.mxgemm(c.lin.w, c.lin.w_scale, codes, scales, 8, 1032, 1024, split_k,
              ws.buf if ws else None, ws.nbytes if ws else 0, plain)
    ids = torch.tensor([-1, 0, -1, 9, 2, -1, 3, 1], dtype=torch.int32, device="cuda")
    got = c.lin(codes, ids, x_scale=scales)
    bare = ((ids < 0) | (ids >= 3)).cpu()
    assert torch.equal(got.cpu()[bare], plain.cpu()[bare])
    assert not torch.equal(got.cpu()[~bare], plain.cpu()[~bare])
    none = c.lin(codes, torch.full_like(ids, -1), x_scale=scales)
    assert torch.equal(none, plain)


def test_zero_adapter_and_special_values(env):
    """A zero B keeps mxgemm's bits; an infinity in one row's x stays there."""
    mx, dv = env
    c = Case(dv, 4, 256, 512, 1, 8, 2, seed=4)
    ids = torch.tensor([0, 1, 0, 1], dtype=torch.int32, device="cuda")
    x = c._bf(c.xb)
    want = c.lin(x, ids).clone()
    bad = x.clone()
    bad[2, 9] = float("inf")
    got = c.lin(bad, ids)
    assert torch.equal(got[[0, 1, 3]], want[[0, 1, 3]]) and not torch.isfinite(got[2]).all()
    none = c.lin(x, torch.full_like(ids, -1)).clone()
    c.lin.b.zero_()
    assert torch.equal(c.lin(x, ids), none)


@pytest.mark.parametrize("split_k", [1, 4])
def test_publish_and_collect(env, split_k):
    """The published product: the plain call's bits with negative zero cleared,
    and an idle mailbox after the collect."""
    mx, dv = env
    from oracle import codecs, mailbox

    c = Case(dv, 5, 1032, 1024, split_k, 16, 3, seed=5)
    ids = torch.tensor([2, -1, 0, 1, 1], dtype=torch.int32, device="cuda")
    mbx = dv.Mailbox(1, 2 * 5 * 1032)
    raw = torch.empty(5, 1032, dtype=torch.bfloat16, device="cuda")
    for call in range(4):
        x = c._bf(c.xb)
        want = c.lin(x, ids).clone()
        c.lin.publish(mbx, x, ids, c_out=raw)
        got = dv.as_u16(dv.collect(mbx, 2 * 5 * 1032)).reshape(5, 1032)
        bits = dv.as_u16(want.view(torch.int16))
        assert np.array_equal(dv.as_u16(raw.view(torch.int16)), bits)
        assert np.array_equal(got, codecs.clear_negative_zero(bits))
        assert not mailbox.check_idle_slots(mbx.slot_words())
    assert mbx.state_words()[mx.STATE_ERROR] == 0


def test_rows_behind(env):
    """Rows behind the last stay as they were."""
    mx, dv = env
    c = Case(dv, 3, 264, 512, 1, 16, 3, seed=6)
    ids = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    x = c._bf(c.xb)
    want = c.lin(x, ids).clone()
    out = torch.full((5, 264), 3.0, dtype=torch.bfloat16, device="cuda")
    c.lin(x, ids, c_out=out[1:4])
    assert torch.equal(out[1:4], want) and (out[[0, 4]] == 3).all()


def test_marked_scratch(env):
    """A scratch with its error word set (as a wait that gave up leaves it): the
    same bits, every workgroup on its own."""
    mx, dv = env
    for split_k, rank in ((1, 24), (4, 24), (1, 128), (4, 128)):
        c = Case(dv, 3, 520, 1024, split_k, rank, 2, seed=9)
        x, ids = c._bf(c.xb), torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
        want = c.lin(x, ids).clone()
        c.lin.scratch[mx.WS_ERROR] = mx.ERR_SPLITK_SPIN
        for _ in range(3):
            assert torch.equal(c.lin(x, ids), want)
        mx.mxgemm_lora_scratch_init(c.lin.scratch, c.lin.scratch_bytes)
        assert torch.equal(c.lin(x, ids), want)


def test_refusals(env):
    mx, dv = env
    c = Case(dv, 4, 256, 512, 1, 8, 2, seed=7)
    x, ids = c._bf(c.xb), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((x.float(), ids), (x[:, :256], ids), (x, ids.long()), (x, ids[:3]),
                (x.repeat(3, 1), ids.repeat(3)), (x.cpu(), ids)):
        with pytest.raises(ValueError):
            c.lin(*bad)
    with pytest.raises(ValueError):
        c.lin(x, ids, x_scale=torch.zeros(4, 16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        dv.AdaptedLinear(torch.from_numpy(c.p.w).cuda(), torch.from_numpy(c.p.ws).cuda(),
                         c.lin.a[:, :4].contiguous(), c.lin.b[:, :, :4].contiguous(), c.lin.scale)
