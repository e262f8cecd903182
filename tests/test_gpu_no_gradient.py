"""The decode operators have no backward pass: what requires a gradient is
refused, and taken under torch.no_grad."""

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


def _refused(call, leaves):
    want = [t.clone() for t in _list(call())]
    for t in leaves:
        t.requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            for u, v in zip(_list(call()), want):
                assert torch.equal(u, v) and not u.requires_grad
        with torch.inference_mode():
            call()
        t.requires_grad_(False)
    for u, v in zip(_list(call()), want):
        assert torch.equal(u, v)


def _list(v):
    return list(v) if isinstance(v, tuple) else [v]


def test_gradients_are_refused(dv):
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = torch.randint(0, 120, (4, 256, 256), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.full((4, 256, 8), 118, dtype=torch.uint8, device="cuda")
    layer = dv.Experts(w, s, w[:, :, :128].contiguous(), s[:, :, :4].contiguous())
    logits, bias, x = new(8, 4), new(4), new(8, 256).bfloat16()
    ids, weights = dv.route(logits, 2, bias=bias)
    _refused(lambda: dv.route(logits, 2, bias=bias), (logits, bias))
    _refused(lambda: layer(x, ids, weights), (x, weights))
    a, b, scale = new(2, 16, 256).bfloat16(), new(2, 256, 16).bfloat16(), new(2)
    rows = torch.arange(8, dtype=torch.int32, device="cuda") % 2
    lin = dv.AdaptedLinear(w[0], s[0], a, b, scale)
    _refused(lambda: lin(x, rows), (x, a, b, scale))
    with pytest.raises(ValueError, match="gradient"):
        dv.AdaptedLinear(w[0], s[0], a.requires_grad_(), b, scale)
    with torch.no_grad():  # a trained stack that serves
        lin = dv.AdaptedLinear(w[0], s[0], a, b, scale)
        lin(x, rows)
