"""The decode operators on a given stream while the current one is busy: their
outputs and the objects' memory are not memory that queued work still uses, and what
the caller drops right after a call stays until the call has read it."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HOLD = 20_000_000  # cycles: some 10 ms


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


def _leave_behind(sizes):
    """Frees blocks of these sizes that the current stream writes a while later."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda._sleep(HOLD)
    for b in blocks:
        b.fill_(0x55)


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    return torch.randn(64, 256, device="cuda", generator=g), g


@pytest.mark.parametrize("raw", [False, True])
def test_fresh_outputs(dv, raw):
    x, g = _inputs()
    w = torch.randint(0, 120, (4, 256, 256), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.full((4, 256, 8), 118, dtype=torch.uint8, device="cuda")
    w2, s2 = w[:, :, :128].contiguous(), s[:, :, :4].contiguous()
    layer = dv.Experts(w, s, w2, s2)
    a = torch.randn(2, 16, 256, device="cuda", generator=g).bfloat16()
    b = torch.randn(2, 256, 16, device="cuda", generator=g).bfloat16()
    lin = dv.AdaptedLinear(w[0], s[0], a, b, torch.ones(2, device="cuda"))
    xb, rows = x.bfloat16(), torch.arange(8, dtype=torch.int32, device="cuda") % 2
    ids, weights = dv.route(x[:, :4], 2)
    want = [*dv.route(x, 8), layer(xb, ids, weights), lin(xb[:8], rows)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = side.cuda_stream if raw else side
    _leave_behind([t.numel() * t.element_size() for t in want])
    got = [*dv.route(x, 8, stream=on), layer(xb, ids, weights, stream=on),
           lin(xb[:8], rows, stream=on)]
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)


@pytest.mark.parametrize("raw", [False, True])
def test_objects_made_on_a_stream(dv, raw):
    x, g = _inputs()
    w = torch.randint(0, 120, (4, 256, 256), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.full((4, 256, 8), 118, dtype=torch.uint8, device="cuda")
    w2, s2 = w[:, :, :128].contiguous(), s[:, :, :4].contiguous()
    a = torch.randn(2, 128, 256, device="cuda", generator=g).bfloat16()
    b = torch.randn(2, 256, 128, device="cuda", generator=g).bfloat16()
    one = torch.ones(2, device="cuda")
    xb, rows = x.bfloat16(), torch.arange(8, dtype=torch.int32, device="cuda") % 2
    ids, weights = dv.route(x[:, :4], 2)
    layer, lin = dv.Experts(w, s, w2, s2, 128), dv.AdaptedLinear(w[0], s[0], a, b, one, 2)
    want = layer(xb, ids, weights), lin(xb[:8], rows)
    sizes = [t.numel() * t.element_size() for t in
             (layer.w13, layer.w13_scale, layer.w2, layer.w2_scale, layer.workspace, lin.w,
              lin.w_scale, lin.scratch, lin.workspace.buf)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = side.cuda_stream if raw else side
    _leave_behind(sizes)
    layer = dv.Experts(w, s, w2, s2, 128, stream=on)
    lin = dv.AdaptedLinear(w[0], s[0], a, b, one, 2, stream=on)
    torch.cuda.synchronize()
    got = layer(xb, ids, weights, stream=on), lin(xb[:8], rows, stream=on)
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    assert lin.errors() == 0


def test_dropped_after_the_call(dv):
    """Inputs, and objects used on another stream than theirs, dropped while that
    stream has not come to the call; the current stream takes their memory."""
    x, g = _inputs()
    w = torch.randint(0, 120, (4, 256, 256), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.full((4, 256, 8), 118, dtype=torch.uint8, device="cuda")
    w2, s2 = w[:, :, :128].contiguous(), s[:, :, :4].contiguous()
    layer, xb = dv.Experts(w, s, w2, s2, 128), x.bfloat16()
    ids, weights = dv.route(x[:, :4], 2)
    want = [*dv.route(x, 8), layer(xb, ids, weights)]
    copies = x.clone(), xb.clone(), ids.clone(), weights.clone()
    sizes = [t.numel() * t.element_size() for t in
             (x, xb, ids, weights, layer.w13, layer.w2, layer.w13_scale, layer.w2_scale)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    x, xb, ids, weights = copies
    del copies
    got = [*dv.route(x, 8, stream=side), layer(xb, ids, weights, stream=side)]
    del x, xb, ids, weights, layer
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in sizes
            for _ in range(3)]
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    del junk


def test_streams_of_another_device_are_refused(dv, monkeypatch):
    class Other:
        device, cuda_stream = torch.device("cuda", 1), 0

    x, _ = _inputs()
    with pytest.raises(ValueError):
        dv.route(x, 4, stream=Other())
