"""mxgemm_lora launches without split-K that share the device: two projections
with more workgroups than it runs, on two streams. The bits of the calls alone, in no
multiple of their time. (A share of u whose workgroup does not run is dealt again
among those that wait for it.)"""

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


@pytest.mark.parametrize("form", ["bf16", "mxfp8"])
def test_two_wide_projections(dv, form):
    g = torch.Generator(device="cuda").manual_seed(1)
    m, k, ids = 8, 4096, torch.arange(8, dtype=torch.int32, device="cuda") % 4
    new = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    lins = []
    for n, rank in ((12288, 64), (11008, 128)):
        w = torch.randint(0, 120, (n, k), dtype=torch.uint8, device="cuda", generator=g)
        s = torch.full((n, k // 32), 118, dtype=torch.uint8, device="cuda")
        lins.append(dv.AdaptedLinear(w, s, new(4, rank, k), new(4, n, rank),
                                     torch.ones(4, device="cuda")))
    if form == "bf16":
        x, xs = new(m, k), None
    else:
        x = torch.randint(0, 120, (m, k), dtype=torch.uint8, device="cuda", generator=g)
        xs = torch.full((m, k // 32), 118, dtype=torch.uint8, device="cuda")
    want = [lin(x, ids, x_scale=xs).clone() for lin in lins]
    outs = [torch.empty_like(v) for v in want]
    streams = [torch.cuda.Stream() for _ in lins]

    def us(on, passes=20):
        best = float("inf")
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            a.record()
            for s in on:
                s.wait_event(a)
            for _ in range(passes):
                for lin, s, out in zip(lins, on, outs):
                    lin(x, ids, x_scale=xs, c_out=out, stream=s)
            for s in on:
                torch.cuda.current_stream().wait_stream(s)
            b.record()
            torch.cuda.synchronize()
            for u, v in zip(outs, want):
                assert torch.equal(u, v)
            best = min(best, 1e3 * a.elapsed_time(b) / passes)
        return best

    one, two = us(streams[:1] * 2), us(streams)
    print(f"{form}: one stream {one:.1f} us a pair, two {two:.1f} us")
    assert two < 2 * one + 50
    assert [lin.errors() for lin in lins] == [0, 0]
