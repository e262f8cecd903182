"""A router, its pairs and the experts' products over a prompt, as they are used together: eager, captured, on two
streams, on a given stream while the current one is busy. Each step is held against the oracle on the results of the
step before it."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as oracle  # noqa: E402
from rows_cases import close, cuda, f64, weights  # noqa: E402

HOLD = 20_000_000  # cycles: some 10 ms
EXPERTS, HIDDEN, INTER, TOP_K = 6, 512, 256, 2


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import device

    torch.cuda.set_device(0)
    return device


@pytest.fixture(scope="module", params=[("mxfp4", "mxfp4"), ("mxfp4", "mxfp8"), ("mxfp8", "mxfp8")],
                ids=lambda p: "-".join(p))
def layer(dv, request):
    rng = np.random.default_rng(8)
    w13 = weights(rng, request.param[0], EXPERTS, 2 * INTER, HIDDEN)
    w2 = weights(rng, request.param[0], EXPERTS, HIDDEN, INTER)
    made = dv.PromptExperts(*map(cuda, (*w13, *w2)), activation=request.param[1])
    return made, w13, w2


def _inputs(tokens, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(tokens, EXPERTS, device="cuda", generator=g),
            torch.randn(tokens, HIDDEN, device="cuda", generator=g).bfloat16())


@pytest.mark.parametrize("tokens", [1, 7, 90, 400])
def test_the_run_of_them(dv, layer, tokens):
    made, w13, w2 = layer
    logits, x = _inputs(tokens, tokens)
    ids, probs = dv.route(logits, TOP_K, renormalize=True)
    ids[0, 0] = -1
    quantize = {4: dv.quantize4, 8: dv.quantize8}[made.up.activation]
    order, offsets = dv.sort_pairs(ids, EXPERTS)
    want = oracle.sort_pairs(ids.cpu().numpy(), EXPERTS)
    assert np.array_equal(order.cpu().numpy(), want[0]) and np.array_equal(offsets.cpu().numpy(), want[1])
    xq, xs = quantize(x)
    h = made.up(xq, xs, offsets, order, gather=TOP_K)
    exact, slack, written = oracle.grouped(*w13, xq.cpu().numpy(), xs.cpu().numpy(), want[1], want[0], TOP_K,
                                           gated=True, rows=TOP_K * tokens)
    assert close(h[cuda(written)], exact[written], slack[written])
    hq, hs = quantize(h)
    y = made.down(hq, hs, offsets, order, scatter=True)
    exact, slack, written = oracle.grouped(*w2, hq.cpu().numpy()[:, :], np.where(hs.cpu().numpy() == 255, 0,
                                           hs.cpu().numpy()), want[1], want[0], scatter=True)
    assert close(y[cuda(written)], exact[written], slack[written])
    out = dv.combine(y, ids, probs, EXPERTS)
    yv = np.where(written[:, None], f64(y), 0.0).reshape(tokens, TOP_K, HIDDEN)
    assert close(out, *oracle.combine(yv, ids.cpu().numpy(), probs.cpu().numpy(), EXPERTS))
    assert torch.equal(made(x, ids, probs), out)


def test_captured_and_replayed(dv, layer):
    made = layer[0]
    logits, x = _inputs(90, 1)

    def step():
        ids, probs = dv.route(logits, TOP_K, renormalize=True)
        return made(x, ids, probs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(2, 6):
        a, b = _inputs(90, seed)
        logits.copy_(a)
        x.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())  # eager work between the replays


def test_two_streams_at_once(dv, layer):
    made = layer[0]
    runs = []
    for seed in (1, 2):
        logits, x = _inputs(300, seed)
        ids, probs = dv.route(logits, TOP_K)
        runs.append((x, ids, probs, made(x, ids, probs)))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, (x, ids, probs, _) in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(made(x, ids, probs))
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert torch.equal(out, runs[i % 2][3])


@pytest.mark.parametrize("raw", [False, True])
def test_on_a_given_stream(dv, layer, raw):
    """Fresh outputs and what a call makes for itself are not memory that queued work of the current stream still
    writes."""
    made = layer[0]
    logits, x = _inputs(90, 3)
    ids, probs = dv.route(logits, TOP_K)
    want = made(x, ids, probs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda")
              for n in (720, 28, 1024, 90 * 512, 90 * 1024, 180 * 512, 180 * 1024, 180 * 8, 90 * 16) for _ in range(3)]
    torch.cuda._sleep(HOLD)
    for b in blocks:
        b.fill_(0x55)
    del blocks, b
    got = made(x, ids, probs, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_what_the_caller_drops(dv, layer):
    made = layer[0]
    logits, x = _inputs(90, 4)
    ids, probs = dv.route(logits, TOP_K)
    want = made(x, ids, probs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    mine = x.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = made(mine, ids, probs, stream=side)
    del mine
    again = torch.full_like(x, 9.0)  # would take the dropped memory
    torch.cuda.synchronize()
    assert torch.equal(got, want) and (again == 9).all()


def test_gradients_are_refused(dv, layer):
    made = layer[0]
    logits, x = _inputs(8, 5)
    ids, probs = dv.route(logits, TOP_K)
    want = made(x, ids, probs)
    for t in (x, probs):
        t.requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            made(x, ids, probs)
        with torch.no_grad():
            assert torch.equal(made(x, ids, probs), want)
        t.requires_grad_(False)


def test_refusals(dv, layer):
    made, w13, w2 = layer
    with pytest.raises(ValueError):
        dv.PromptExperts(*map(cuda, (*w13, w13[0], w13[1])))
    _, x = _inputs(8, 5)
    ids = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        made(x[:7], ids, torch.zeros(7, 2, device="cuda"))
