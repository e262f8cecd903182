"""mxgemm_lora where the projection has more workgroups than the device runs at
once, without split-K: against the float64 oracle, and in time."""

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


def _us(call, passes=10):
    """The fastest of five runs, per call."""
    best = float("inf")
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        for _ in range(passes):
            call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b) / passes)
    return best


@pytest.mark.parametrize("m,n,k,rank,adapters", [
    (4, 12288, 4096, 64, 2), (8, 11008, 4096, 32, 5), (8, 9216, 4096, 128, 3),
    (2, 20480, 4096, 64, 1),
])
def test_many_workgroups(env, m, n, k, rank, adapters):
    """u's dot products are dealt to workgroups that run: the adapters cost no
    multiple of the projection. (Where half of the products waited for workgroups that
    could not start, every workgroup computed all of them alone.)"""
    from test_gpu_adapters import Case

    mx, dv = env
    c = Case(dv, m, n, k, 1, rank, adapters)
    ids = c.rng.integers(0, adapters, m)
    c.check(ids)
    x, xs = torch.from_numpy(c.p.x).cuda(), torch.from_numpy(c.p.xs).cuda()
    dev_ids = torch.from_numpy(np.asarray(ids, dtype=np.int32)).cuda()
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    plain = _us(lambda: mx.mxgemm(c.lin.w, c.lin.w_scale, x, xs, m, n, k, 1, None, 0, out))
    adapted = _us(lambda: c.lin(x, dev_ids, x_scale=xs, c_out=out))
    print(f"m={m} n={n} k={k} rank={rank}: mxgemm {plain:.1f} us, with adapters {adapted:.1f} us")
    assert adapted < 2 * plain + 10


@pytest.mark.parametrize("m,n,k,split_k,rank", [(5, 4096, 16384, 8, 32), (1, 32768, 4096, 1, 128)])
def test_many_workgroups_bf16(env, m, n, k, split_k, rank):
    """BF16 x on tiles of five waves, of whose workgroups two would fit a CU by the
    sum of its registers, but not by SIMD: in time, against the same call without
    adapters in the rows."""
    mx, dv = env
    g = torch.Generator(device="cuda").manual_seed(n)
    codes = torch.randint(0, 120, (n, k), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.full((n, k // 32), 118, dtype=torch.uint8, device="cuda")
    a = torch.randn(4, rank, k, device="cuda", generator=g).bfloat16()
    b = torch.randn(4, n, rank, device="cuda", generator=g).bfloat16()
    lin = dv.AdaptedLinear(codes, scales, a, b, torch.ones(4, device="cuda"), split_k)
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    ids = torch.arange(m, dtype=torch.int32, device="cuda") % 4
    none = torch.full_like(ids, -1)
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    bare = _us(lambda: lin(x, none, c_out=out))
    adapted = _us(lambda: lin(x, ids, c_out=out))
    print(f"m={m} n={n} k={k} split_k={split_k} rank={rank}: none {bare:.1f} us, adapters "
          f"{adapted:.1f} us")
    assert adapted < 2 * bare + 10
