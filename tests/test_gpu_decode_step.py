"""The per-row decode operators together, as a decode step uses them (on an
MI355X): projection with adapters -> publish -> collect -> router logits by the
plain GEMM -> route -> experts -> publish -> collect. Every stage is checked
against the oracle on the bits it was given; the whole step, captured into a
graph and replayed with new inputs, gives the eager call's bits; operators on
two streams at once keep theirs. The tests of one adapter scratch under several
streams and graphs are here too: streams share a few hardware queues, and the
all-gather whose peers publish on another stream needs two that do not, so no
test that makes streams comes before it."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

M, K, HIDDEN, EXPERTS, INTER, RANK, ADAPTERS, TOP_K = 5, 2048, 1024, 32, 256, 16, 3, 4


@pytest.fixture(scope="module")
def env():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    from mxfp8_decode_gemm_amd import binding, device

    torch.cuda.set_device(0)
    return binding, device


def _bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _mx(rng, *shape):
    from workloads import generate

    v = rng.standard_normal((int(np.prod(shape[:-1])), shape[-1])) * shape[-1] ** -0.5
    q, s = generate.quantize_mxfp8(v)
    return q.reshape(shape), s.reshape(*shape[:-1], shape[-1] // 32)


class Step:
    """One layer's decode step on fixed buffers."""

    def __init__(self, env, seed, split_k):
        mx, dv = self.mx, self.dv = env
        from workloads import generate

        rng = np.random.default_rng(seed)
        self.w, self.ws = _mx(rng, HIDDEN, K)
        self.a = generate.bf16_bits((rng.standard_normal((ADAPTERS, RANK, K)) * K**-0.5)
                                    .astype(np.float32))
        self.b = generate.bf16_bits(rng.standard_normal((ADAPTERS, HIDDEN, RANK))
                                    .astype(np.float32))
        self.scale = rng.uniform(0.5, 1.5, ADAPTERS).astype(np.float32)
        self.moe = (*_mx(rng, EXPERTS, 2 * INTER, HIDDEN), *_mx(rng, EXPERTS, HIDDEN, INTER))
        cuda = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
        self.lin = dv.AdaptedLinear(cuda(self.w), cuda(self.ws), _bf(self.a), _bf(self.b),
                                    cuda(self.scale), split_k)
        self.experts = dv.Experts(*(cuda(v) for v in self.moe), M * TOP_K)
        gate, gate_s = _mx(rng, EXPERTS, HIDDEN)
        self.gate = dv.pack_weight(cuda(gate), cuda(gate_s), EXPERTS, HIDDEN)
        self.bias = cuda((0.05 * rng.standard_normal(EXPERTS)).astype(np.float32))
        self.boxes = [dv.Mailbox(1, 2 * M * HIDDEN) for _ in range(2)]
        new = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.ids = new(M, K), new(M, t=torch.int32)
        self.y, self.out, self.z = new(M, HIDDEN), new(M, HIDDEN), new(M, HIDDEN)
        self.q, self.qs = new(M, HIDDEN, t=torch.uint8), new(M, HIDDEN // 32, t=torch.uint8)
        self.logits = new(M, EXPERTS)
        self.chosen = new(M, TOP_K, t=torch.int32)
        self.weights = new(M, TOP_K, t=torch.float32)
        self.mask = torch.zeros(M, EXPERTS, dtype=torch.bfloat16, device="cuda")

    def set(self, seed):
        from workloads import generate

        rng = np.random.default_rng(seed)
        self.x.copy_(_bf(generate.bf16_bits(rng.standard_normal((M, K)).astype(np.float32))))
        self.ids.copy_(torch.from_numpy(rng.integers(-1, ADAPTERS, M).astype(np.int32)))
        self.mask.zero_()
        self.mask[seed % M] = -torch.inf  # a row without any expert
        self.mask[(seed + 1) % M, 2:] = -torch.inf  # one with fewer than top_k

    def run(self):
        mx, dv = self.mx, self.dv
        self.lin.publish(self.boxes[0], self.x, self.ids)
        mx.mailbox_collect_sum(self.boxes[0].mb, self.y, 2 * M * HIDDEN)
        mx.mxfp8_quantize(self.y, M, HIDDEN, self.q, self.qs)
        mx.mxgemm(*self.gate, self.q, self.qs, M, EXPERTS, HIDDEN, 1, None, 0, self.logits)
        self.logits.add_(self.mask)
        dv.route(self.logits, TOP_K, score="sigmoid", bias=self.bias, groups=4, top_groups=2,
                 group_best=2, renormalize=True, scale=2.0, ids=self.chosen, weights=self.weights)
        self.experts(self.y, self.chosen, self.weights, out=self.out)
        mx.mailbox_publish(self.boxes[1].mb, 0, self.out, 2 * M * HIDDEN)
        mx.mailbox_collect(self.boxes[1].mb, self.z, 2 * M * HIDDEN)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.y, self.logits, self.chosen, self.weights, self.out,
                                    self.z)]

    def check(self):
        from oracle import decode, gemm, quant

        torch.cuda.synchronize()
        x = _f64(self.x)
        codes, scales = quant.quantize_bf16(
            self.x.view(torch.int16).cpu().numpy().view(np.uint16))
        up = lambda b: (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)  # noqa: E731
        exact, bound = decode.adapted(gemm.dequantize(codes, scales), x, self.w, self.ws,
                                      up(self.a), up(self.b), self.scale.astype(np.float64),
                                      self.ids.cpu().numpy())
        assert (np.abs(_f64(self.y) - exact) <= bound).all()
        want, w = decode.route(_f64(self.logits), TOP_K, "sigmoid", self.bias.cpu().numpy(), 4, 2,
                               2, True, 2.0)
        ids = self.chosen.cpu().numpy()
        assert np.array_equal(ids, want)
        # (the weight bound of the router's own tests, logits of order one)
        assert (np.abs(_f64(self.weights) - w) <= 2.0**-24 * 160 * np.abs(w)).all()
        assert (ids == -1).any()
        exact, bound = decode.experts(_f64(self.y), ids, self.weights.cpu().numpy(), *self.moe)
        assert (np.abs(_f64(self.out) - exact) <= bound).all()
        assert torch.equal(self.z, self.out + 0.0)  # negative zero cleared
        for box in self.boxes:
            assert box.state_words()[self.mx.STATE_ERROR] == 0


@pytest.mark.parametrize("split_k", [1, 4])
def test_step(env, split_k):
    step = Step(env, 1, split_k)
    for seed in (1, 2, 3):
        step.set(seed)
        step.run()
        step.check()


@pytest.mark.parametrize("split_k", [1, 4])
def test_step_captured(env, split_k):
    """Replays with other inputs, with eager steps and synchronizations between."""
    step, eager = Step(env, 2, split_k), Step(env, 2, split_k)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for s in (step, eager):
            s.set(0)
            s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.run()
    for seed in range(4, 9):
        step.set(seed)
        eager.set(seed)
        torch.cuda.synchronize()
        graph.replay()
        got = step.results()
        eager.run()
        for g, w in zip(got, eager.results()):
            assert torch.equal(g, w)
    step.check()


def test_two_streams(env):
    """Steps of two layers (without split-K) on two streams at once."""
    steps = [Step(env, s, 1) for s in (3, 4)]
    want = []
    for s in steps:
        s.set(7)
        s.run()
        want.append(s.results())
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(8):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
    for s, w in zip(steps, want):
        for a, b in zip(s.results(), w):
            assert torch.equal(a, b)


def test_another_device_is_refused(env, monkeypatch):
    """A call whose tensors are not on the current device."""
    mx, dv = env
    step = Step(env, 5, 1)
    step.set(1)
    monkeypatch.setattr(dv, "_device", lambda: 1)
    with pytest.raises(ValueError):
        dv.route(step.logits, TOP_K)
    with pytest.raises(ValueError):
        step.experts(step.y, step.chosen, step.weights)
    with pytest.raises(ValueError):
        step.lin(step.x, step.ids)


def test_one_scratch_for_projections_captured(env):
    """Projections of other sizes (with helping workgroups, and more workgroups
    than flag words of a small one) in one graph on one scratch: replays with
    other activations, eager calls between, each against a scratch of its own."""
    from test_gpu_adapters import Case

    mx, dv = env
    cases = [Case(dv, 8, 64, 4096, 1, 128, 4, seed=21), Case(dv, 8, 40960, 128, 1, 128, 4, seed=22),
             Case(dv, 8, 1032, 1024, 4, 64, 4, seed=23)]
    own = [(c.lin.scratch, c.lin.scratch_bytes) for c in cases]
    ids = torch.tensor([3, 0, -1, 2, 0, 1, 1, 3], dtype=torch.int32, device="cuda")
    xs = [c._bf(c.xb) for c in cases]
    outs = [torch.empty(8, c.p.n, dtype=torch.bfloat16, device="cuda") for c in cases]

    def share(shared):
        for c, (scratch, nbytes) in zip(cases, own):
            c.lin.scratch, c.lin.scratch_bytes = own[1] if shared else (scratch, nbytes)

    def step():
        for c, x, out in zip(cases, xs, outs):
            c.lin(x, ids, c_out=out)

    share(True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(4):
        for x in xs:
            x.copy_(x.roll(1, 0) * (1 + replay))
        ids.copy_(ids.roll(1))
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone() for out in outs]
        share(False)
        step()
        torch.cuda.synchronize()
        share(True)
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
        step()  # eager, on the shared one


def test_one_scratch_for_calls_of_all_sizes(env):
    """The epoch keeps a call from taking an earlier one's pairs: other rows,
    ids and values through one scratch, on two streams in order."""
    from test_gpu_adapters import Case

    mx, dv = env
    c = Case(dv, 8, 1032, 1024, 4, 16, 3, seed=8)
    side = torch.cuda.Stream()
    x = c._bf(c.xb)
    rng = np.random.default_rng(1)
    for call in range(12):
        m = int(rng.integers(1, 9))
        ids = torch.from_numpy(rng.integers(-1, 3, m).astype(np.int32)).cuda()
        rows = torch.from_numpy(rng.permutation(8)[:m]).cuda()
        part = x[rows].contiguous()
        torch.cuda.synchronize()
        with torch.cuda.stream(side if call % 2 else torch.cuda.default_stream()):
            got = c.lin(part, ids)
        torch.cuda.synchronize()
        fresh = dv.AdaptedLinear(torch.from_numpy(c.p.w).cuda(), torch.from_numpy(c.p.ws).cuda(),
                                 c.lin.a, c.lin.b, c.lin.scale, 4)
        assert torch.equal(got, fresh(part, ids))
