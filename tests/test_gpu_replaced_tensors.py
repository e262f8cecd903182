"""dv.AdaptedLinear and dv.Experts whose tensors the caller replaces: the
adapters, the scratch, and what may not be replaced."""

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


def _fresh(dv, c, split_k=1):
    return dv.AdaptedLinear(torch.from_numpy(c.p.w).cuda(), torch.from_numpy(c.p.ws).cuda(),
                            c.lin.a, c.lin.b, c.lin.scale, split_k)


def _stack(seed, adapters, n, k, rank):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return (new(adapters, rank, k) * k**-0.5).bfloat16(), new(adapters, n, rank).bfloat16(), new(
        adapters)


def test_replaced_adapters(env):
    """Other tensors, of other ranks and counts, by assignment and as .data; the old
    ones' memory is written over."""
    from test_gpu_adapters import Case

    mx, dv = env
    n, k = 264, 512
    c = Case(dv, 3, n, k, 1, 16, 3, seed=31)
    x = c._bf(c.xb)
    ids = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    wide = torch.tensor([4, 1, 0], dtype=torch.int32, device="cuda")
    c.lin(x, ids)
    for seed, adapters, rank in ((1, 3, 16), (2, 5, 32), (3, 1, 8), (4, 5, 32)):
        c.lin.a, c.lin.b, c.lin.scale = _stack(seed, adapters, n, k, rank)
        junk = [torch.full((4096,), 1e9, device="cuda") for _ in range(16)]
        got = c.lin(x, wide)
        assert torch.equal(got, _fresh(dv, c)(x, wide)) and torch.isfinite(got).all()
        del junk
    a, b, scale = _stack(5, 5, n, k, 32)
    c.lin.a.data, c.lin.b.data, c.lin.scale.data = a, b, scale
    del a, b, scale
    junk = [torch.full((4096,), 1e9, device="cuda") for _ in range(16)]
    assert torch.equal(c.lin(x, wide), _fresh(dv, c)(x, wide))
    del junk
    c.lin.a = c.lin.a[:2]  # the same address, fewer adapters
    with pytest.raises(ValueError):
        c.lin(x, wide)
    c.lin.b, c.lin.scale = c.lin.b[:2], c.lin.scale[:2]
    assert torch.equal(c.lin(x, wide), _fresh(dv, c)(x, wide))
    for bad in (c.lin.a.float(), c.lin.a[:, :12].contiguous(), c.lin.a.cpu(), None):
        good, c.lin.a = c.lin.a, bad
        with pytest.raises((ValueError, AttributeError)):
            c.lin(x, wide)
        c.lin.a = good
    assert torch.equal(c.lin(x, wide), _fresh(dv, c)(x, wide))


def test_written_adapters(env):
    """Writes in place are seen by the next call and the next replay."""
    from test_gpu_adapters import Case

    mx, dv = env
    c = Case(dv, 4, 520, 1024, 1, 16, 2, seed=32)
    x, ids = c._bf(c.xb), torch.tensor([0, 1, -1, 1], dtype=torch.int32, device="cuda")
    out = torch.empty(4, 520, dtype=torch.bfloat16, device="cuda")
    c.lin(x, ids, c_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.lin(x, ids, c_out=out)
    for step in range(3):
        for t, v in zip((c.lin.a, c.lin.b, c.lin.scale), _stack(step, 2, 520, 1024, 16)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _fresh(dv, c)(x, ids)) and torch.equal(c.lin(x, ids), out)


def test_what_may_not_be_replaced(env):
    from test_gpu_adapters import Case
    from test_gpu_experts import Layer

    mx, dv = env
    c = Case(dv, 3, 264, 512, 2, 16, 3, seed=33)
    for name in ("w", "w_scale", "workspace"):
        with pytest.raises(AttributeError):
            setattr(c.lin, name, None)
    small = torch.zeros(mx.mxgemm_lora_scratch_bytes(8) // 4, dtype=torch.int32, device="cuda")
    big = dv.AdaptedLinear(torch.zeros(40960, 128, dtype=torch.uint8, device="cuda"),
                           torch.zeros(40960, 4, dtype=torch.uint8, device="cuda"),
                           *_stack(1, 1, 40960, 128, 8))
    for bad in (small, small.float(), small.cpu(), None):
        with pytest.raises(ValueError):
            big.scratch = bad
    with pytest.raises(ValueError):
        c.lin.scratch_bytes = c.lin.scratch_bytes + 16
    layer = Layer(dv, 34, 3, 128, 128).layer
    for name in ("w13", "w13_scale", "w2", "w2_scale", "workspace"):
        with pytest.raises(AttributeError):
            setattr(layer, name, None)
