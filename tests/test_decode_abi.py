"""include/mxdecode.h without a GPU: the library exports what it declares, its
constants match the binding, sizes, and the refusals of bad arguments on the
host before any HIP call."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mx():
    from mxfp8_decode_gemm_amd import build as b

    if not os.path.exists(b.LIB):
        b.build()
    from mxfp8_decode_gemm_amd import binding

    return binding


def test_exports_every_declared_function(mx):
    names = mx.header_functions(mx.DECODE_HEADER_PATH)
    assert names == ["mxgemm_lora", "mxgemm_lora_scratch_bytes",
                     "mxgemm_lora_scratch_init", "mxmoe_experts",
                     "mxmoe_pack_weight", "mxmoe_packed_scale_bytes", "mxmoe_packed_weight_bytes",
                     "mxmoe_route", "mxmoe_workspace_bytes"]
    assert not [n for n in names if not hasattr(mx.library(), n) or not hasattr(mx, n)]


def test_constants_and_structures(mx):
    with open(mx.DECODE_HEADER_PATH) as f:
        h = f.read()
    for name in ("ROUTE_SOFTMAX", "ROUTE_SIGMOID", "F32", "BF16", "ROUTE_MAX_EXPERTS",
                 "ROUTE_MAX_GROUPS", "ROUTE_MAX_TOP_K", "MOE_MAX_EXPERTS", "MOE_MAX_PAIRS",
                 "LORA_MAX_RANK"):
        line = [ln for ln in h.splitlines() if ln.startswith(f"#define MXG_{name} ")]
        assert len(line) == 1 and int(line[0].split()[2]) == getattr(mx, name)
    assert ctypes.sizeof(mx.mxmoe_router) == 32 and mx.mxmoe_router.scale.offset == 28
    assert ctypes.sizeof(mx.mxg_lora) == 40 and mx.mxg_lora.rank.offset == 36


def test_sizes(mx):
    assert mx.mxmoe_packed_weight_bytes(3, 256, 128) == 3 * mx.mxgemm_packed_weight_bytes(256, 128)
    assert mx.mxmoe_packed_scale_bytes(3, 256, 128) == 3 * mx.mxgemm_packed_scale_bytes(256, 128)
    for bad in ((0, 256, 128), (1025, 256, 128), (1, 24, 128), (1, 256, 96)):
        assert mx.mxmoe_packed_weight_bytes(*bad) == 0
        assert mx.mxmoe_packed_scale_bytes(*bad) == 0
    # at least h in two BF16 parts and y in FP32 for every pair
    assert mx.mxmoe_workspace_bytes(8, 8, 64, 7168, 2048) >= 64 * 4 * (7168 + 2048)
    # and more for more pairs, whatever the shape of the call
    sizes = [mx.mxmoe_workspace_bytes(p, 1, 24, 256, 384) for p in range(1, 1025)]
    assert sizes == sorted(sizes) and mx.mxmoe_workspace_bytes(16, 8, 24, 256, 384) == sizes[127]
    for bad in ((0, 8, 4, 128, 128), (129, 8, 4, 128, 128), (1, 0, 4, 128, 128),
                (1, 1, 0, 128, 128), (1, 1, 1025, 128, 128), (1, 1, 4, 192, 128),
                (1, 1, 4, 128, 64), (1, 1, 4, 32896, 128), (1, 1, 4, 128, 32896),
                (1 << 30, 4, 4, 128, 128)):
        assert mx.mxmoe_workspace_bytes(*bad) == 0
    # header, an epoch word per workgroup, 1024 pairs
    assert mx.mxgemm_lora_scratch_bytes(8) == 256 + 2048 * 4 + 1024 * 8
    assert mx.mxgemm_lora_scratch_bytes(1 << 20) == 256 + (1 << 16) * 4 + 1024 * 8
    for bad in (0, 12, -8):
        assert mx.mxgemm_lora_scratch_bytes(bad) == 0
    lib = mx.library()
    assert lib.mxgemm_lora_scratch_init(None, 1 << 20, None) == -1
    assert lib.mxgemm_lora_scratch_init(4096, 1024, None) == -1
    assert lib.mxgemm_lora_scratch_init(4096, (1 << 20) + 8, None) == -1
    assert lib.mxgemm_lora_scratch_init(4104, 1 << 20, None) == -2


@pytest.mark.parametrize("kw,code", [
    (dict(experts=0), -1), (dict(experts=1025), -1), (dict(score=2), -1), (dict(score=-1), -1),
    (dict(groups=0), -1), (dict(groups=3), -1), (dict(groups=128, experts=128), -1),
    (dict(top_groups=0), -1), (dict(groups=4, top_groups=5), -1), (dict(group_best=0), -1),
    (dict(group_best=3), -1), (dict(renormalize=2), -1), (dict(top_k=0), -1), (dict(top_k=33), -1),
    (dict(groups=16, top_groups=1, top_k=5), -1), (dict(tokens=0), -1),
    (dict(tokens=(1 << 24) + 1), -1), (dict(row_stride=63), -1), (dict(kind=2), -1),
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(router=None), -1),
    (dict(logits=4098), -2), (dict(kind=1, logits=4097), -2), (dict(bias=4098), -2),
    (dict(ids=4097), -2), (dict(weights=4102), -2),
])
def test_route_refusals(mx, kw, code):
    a = dict(experts=64, top_k=4, score=0, groups=1, top_groups=1, group_best=1, renormalize=1,
             tokens=2, row_stride=None, kind=0, logits=4096, bias=None, ids=4096, weights=4096,
             router=True)
    a.update(kw)
    r = mx.mxmoe_router(a["experts"], a["top_k"], a["score"], a["groups"], a["top_groups"],
                        a["group_best"], a["renormalize"], 1.0)
    rc = mx.library().mxmoe_route(ctypes.byref(r) if a["router"] else None, a["logits"], a["kind"],
                                  a["row_stride"] or a["experts"], a["bias"], a["tokens"],
                                  a["ids"], a["weights"], None)
    assert rc == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), -1), (dict(top_k=0), -1), (dict(tokens=513), -1), (dict(experts=0), -1),
    (dict(experts=1025), -1), (dict(hidden=192), -1), (dict(inter=0), -1), (dict(inter=32896), -1),
    (dict(x=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(w13=None), -1),
    (dict(w13s=None), -1), (dict(w2=None), -1), (dict(w2s=None), -1), (dict(out=None), -1),
    (dict(x=4104), -2), (dict(ids=4098), -2), (dict(weights=4098), -2), (dict(w13=4104), -2),
    (dict(w13s=4104), -2), (dict(w2=4104), -2), (dict(w2s=4104), -2), (dict(out=4104), -2),
    (dict(ws=None), -4), (dict(ws_bytes=16), -4), (dict(ws=4104), -2),
])
def test_experts_refusals(mx, kw, code):
    a = dict(x=4096, ids=4096, weights=4096, w13=4096, w13s=4096, w2=4096, w2s=4096, tokens=4,
             top_k=2, experts=8, hidden=256, inter=128, ws=4096, ws_bytes=1 << 20, out=4096)
    a.update(kw)
    rc = mx.library().mxmoe_experts(*a.values(), None)
    assert rc == code


def test_expert_pack_refusals(mx):
    lib = mx.library()
    ok = [4096, 4096, 2, 32, 128, 4096, 4096, None]
    for i, v, code in ((0, None, -1), (1, None, -1), (5, None, -1), (6, None, -1), (2, 0, -1),
                       (2, 1025, -1), (3, 24, -1), (4, 64, -1), (0, 4104, -2), (1, 4104, -2),
                       (5, 4104, -2), (6, 4104, -2)):
        a = list(ok)
        a[i] = v
        assert lib.mxmoe_pack_weight(*a) == code


@pytest.mark.parametrize("kw,code", [
    (dict(lora=None), -1), (dict(a=None), -1), (dict(b=None), -1), (dict(scale=None), -1),
    (dict(ids=None), -1), (dict(adapters=0), -1), (dict(rank=0), -1), (dict(rank=12), -1),
    (dict(rank=136), -1), (dict(m=0), -1), (dict(m=9), -1), (dict(n=12), -1), (dict(k=96), -1),
    (dict(split_k=3), -1), (dict(c_out=None), -1), (dict(x_bf16=None), -1), (dict(x=4096), -1),
    (dict(x=4096, x_bf16=None), -1), (dict(w=None), -1), (dict(w_scale=None), -1),
    (dict(a=4104), -2), (dict(b=4104), -2), (dict(scale=4098), -2), (dict(ids=4098), -2),
    (dict(x_bf16=4104), -2), (dict(c_out=4104), -2), (dict(scratch=None), -4),
    (dict(scratch_bytes=32), -4), (dict(scratch=4104), -2), (dict(split_k=2), -4),
    (dict(split_k=2, ws=4096, ws_bytes=100), -4), (dict(split_k=2, ws=4104, ws_bytes=1 << 20), -2),
])
def test_lora_refusals(mx, kw, code):
    a = dict(w=4096, w_scale=4096, x=None, x_scale=None, x_bf16=4096, m=2, n=256, k=512, split_k=1,
             ws=None, ws_bytes=0, scratch=4096, scratch_bytes=1 << 16, c_out=4096, a=4096, b=4096,
             scale=4096, ids=4096, adapters=2, rank=16, lora=True)
    a.update(kw)
    lora = mx.mxg_lora(a["a"], a["b"], a["scale"], a["ids"], a["adapters"], a["rank"])
    rc = mx.library().mxgemm_lora(None, a["w"], a["w_scale"], a["x"], a["x_scale"], a["x_bf16"],
                                  a["m"], a["n"], a["k"], a["split_k"], a["ws"], a["ws_bytes"],
                                  ctypes.byref(lora) if a["lora"] else None, a["scratch"],
                                  a["scratch_bytes"], a["c_out"], None)
    assert rc == code


def test_lora_mailbox_capacity(mx):
    """The mailbox rules of mxgemm_publish hold: 2 m n above the slot."""
    mb = mx.mxg_mailbox()
    mb.slots, mb.state, mb.ranks, mb.rank, mb.capacity_bytes = 4096, 8192, 1, 0, 512
    lora = mx.mxg_lora(4096, 4096, 4096, 4096, 2, 16)
    rc = mx.library().mxgemm_lora(ctypes.byref(mb), 4096, 4096, None, None, 4096, 2, 256, 512, 1,
                                  None, 0, ctypes.byref(lora), 4096, 1 << 16, None, None)
    assert rc == -3


def test_device_wrappers_refuse_host_tensors(mx):
    """The torch wrappers look at types, shapes and places before any call."""
    torch = pytest.importorskip("torch")
    from mxfp8_decode_gemm_amd import device as dv

    with pytest.raises(ValueError):
        dv.route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError):
        dv.Experts(torch.zeros(2, 256, 128, dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError):
        dv.AdaptedLinear(torch.zeros(256, 128, dtype=torch.uint8), None, None, None, None)
