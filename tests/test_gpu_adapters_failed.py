"""mxgemm_lora on a split-K workspace whose exchange has failed: nothing that
looks like a result, the bits say so, and arming makes it good."""

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


@pytest.mark.parametrize("n,split_k,rank", [(520, 4, 24), (1032, 8, 128), (64, 2, 128)])
def test_marked_workspace(env, n, split_k, rank):
    from test_gpu_adapters import Case

    mx, dv = env
    c = Case(dv, 3, n, 2048, split_k, rank, 2, seed=11)
    x, ids = c._bf(c.xb), torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    want = c.lin(x, ids).clone()
    assert c.lin.errors() == 0
    c.lin.workspace.buf[mx.WS_ERROR] = mx.ERR_SPLITK_SPIN
    out = torch.full((5, n), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        c.lin(x, ids, c_out=out[1:4])
        assert torch.isnan(out[1:4]).all() and (out[[0, 4]] == 3).all()
    assert torch.isnan(c.lin(x, ids)).all()
    assert c.lin.errors() == mx.ERR_SPLITK_SPIN
    box = dv.Mailbox(1, 2 * 3 * n)
    box.spin_limit = 64
    c.lin.publish(box, x, ids)  # nothing
    dv.collect(box, 2 * 3 * n)
    assert box.state_words()[mx.STATE_ERROR] == mx.ERR_COLLECT_SPIN
    c.lin.rearm()
    for _ in range(2):
        assert torch.equal(c.lin(x, ids), want)
    assert c.lin.errors() == 0


def test_errors_of_the_scratch(env):
    """A marked scratch alone: right results, and the bits."""
    from test_gpu_adapters import Case

    mx, dv = env
    for split_k in (1, 4):
        c = Case(dv, 3, 520, 1024, split_k, 24, 2, seed=12)
        x, ids = c._bf(c.xb), torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
        want = c.lin(x, ids).clone()
        c.lin.scratch[mx.WS_ERROR] = mx.ERR_SPLITK_SPIN
        assert torch.equal(c.lin(x, ids), want) and c.lin.errors() == mx.ERR_SPLITK_SPIN
        c.lin.rearm()
        assert torch.equal(c.lin(x, ids), want) and c.lin.errors() == 0
