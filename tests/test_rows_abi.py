"""include/mxrows.h without a GPU: the library exports what it declares, its constants match the binding, sizes, and the
refusals of bad arguments on the host before any HIP call."""

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
    names = mx.header_functions(mx.ROWS_HEADER_PATH)
    assert names == ["mxfp4_dequantize", "mxfp4_quantize", "mxmoe_combine", "mxmoe_grouped", "mxmoe_sort",
                     "mxmoe_sort_workspace_bytes", "mxrows_pack_weight", "mxrows_packed_scale_bytes",
                     "mxrows_packed_weight_bytes", "mxrows_product", "mxrows_workspace_bytes"]
    assert not [n for n in names if not hasattr(mx.library(), n) or not hasattr(mx, n)]


def test_constants_and_structures(mx):
    with open(mx.ROWS_HEADER_PATH) as f:
        h = f.read()
    for name in ("F16", "MXFP4", "MXFP8", "ROWS_MAX", "ROWS_MAX_N", "ROWS_MAX_K"):
        line = [ln for ln in h.splitlines() if ln.startswith(f"#define MXG_{name} ")]
        assert len(line) == 1 and int(line[0].split()[2]) == getattr(mx, name)
    assert ctypes.sizeof(mx.mxrows_weight) == 40 and mx.mxrows_weight.gated.offset == 32


def test_sizes(mx):
    for f, unit in ((mx.MXFP4, 2048), (mx.MXFP8, 4096)):
        assert mx.mxrows_packed_weight_bytes(f, 3, 64, 256) == 3 * 2 * 2 * unit
        assert mx.mxrows_packed_weight_bytes(f, 1, 40, 128) == 2 * 2 * unit  # n to 64, k to 256
        assert mx.mxrows_packed_scale_bytes(f, 3, 64, 512) == 3 * 2 * 2 * 256
        big = mx.mxrows_packed_weight_bytes(f, 1024, 1 << 20, 65536)
        assert big == 1024 * (1 << 20) * 65536 * unit // 4096
    for bad in ((3, 1, 64, 256), (4, 0, 64, 256), (4, 1025, 64, 256), (4, 1, 0, 256), (4, 1, 12, 256), (4, 1, 64, 0),
                (4, 1, 64, 192), (8, 1, (1 << 20) + 8, 256), (8, 1, 64, 65664), (4, 1, -8, 256)):
        assert mx.mxrows_packed_weight_bytes(*bad) == 0 and mx.mxrows_packed_scale_bytes(*bad) == 0
    assert mx.mxmoe_sort_workspace_bytes(512, 8, 1024) == 0 < mx.mxmoe_sort_workspace_bytes(513, 8, 1)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 33, 64), (1, 1, 0), (1, 1, 1025), ((1 << 24) + 1, 1, 4), (1 << 23, 3, 4)):
        assert mx.mxmoe_sort_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(xq=None), -1), (dict(xs=None), -1), (dict(kind=3), -1), (dict(kind=-1), -1),
    (dict(rows=0), -1), (dict(rows=(1 << 24) + 1), -1), (dict(k=0), -1), (dict(k=48), -1), (dict(k=65568), -1),
    (dict(stride=56), -1), (dict(stride=(1 << 31) + 8), -1), (dict(stride=68), -1), (dict(kind=0, stride=66), -1),
    (dict(x=4104), -2), (dict(xq=4104), -2),
])
def test_quantize_refusals(mx, kw, code):
    a = dict(x=4096, kind=1, stride=64, rows=2, k=64, xq=4096, xs=4096)
    a.update(kw)
    assert mx.library().mxfp4_quantize(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(xq=None), -1), (dict(xs=None), -1), (dict(y=None), -1), (dict(kind=4), -1), (dict(rows=0), -1),
    (dict(k=16), -1), (dict(k=65568), -1), (dict(xq=4100), -2), (dict(y=4104), -2),
])
def test_dequantize_refusals(mx, kw, code):
    a = dict(xq=4096, xs=4096, rows=2, k=64, kind=1, y=4096)
    a.update(kw)
    assert mx.library().mxfp4_dequantize(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(f=1), -1), (dict(w=None), -1), (dict(ws=None), -1), (dict(wp=None), -1), (dict(wsp=None), -1),
    (dict(e=0), -1), (dict(n=12), -1), (dict(k=64), -1), (dict(w=4104), -2), (dict(ws=4098), -2), (dict(wp=4104), -2),
    (dict(wsp=4104), -2),
])
def test_pack_refusals(mx, kw, code):
    a = dict(f=4, w=4096, ws=4096, e=1, n=64, k=256, wp=4096, wsp=4096)
    a.update(kw)
    assert mx.library().mxrows_pack_weight(*a.values(), None) == code


WEIGHT = dict(w=4096, scale=4096, format=4, experts=1, n=64, k=256, gated=0)
BAD_WEIGHTS = [
    (dict(w=None), -1), (dict(scale=None), -1), (dict(format=5), -1), (dict(experts=0), -1), (dict(n=4), -1),
    (dict(k=64), -1), (dict(gated=2), -1), (dict(n=96, gated=1), -1), (dict(w=4104), -2), (dict(scale=4104), -2),
    (dict(format=8), -5),  # on MXFP4 x
]


@pytest.mark.parametrize("wkw,kw,code", [(w, {}, c) for w, c in BAD_WEIGHTS] + [({}, kw, c) for kw, c in [
    (dict(weight=False), -1), (dict(f=6), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(rows=0), -1),
    (dict(rows=(1 << 24) + 1), -1), (dict(out=None), -1), (dict(x=4104), -2), (dict(xs=4098), -2), (dict(out=4104), -2),
]] + [(dict(experts=2), {}, -1)])
def test_product_refusals(mx, wkw, kw, code):
    a = dict(weight=True, f=4, x=4096, xs=4096, rows=2, ws=None, nbytes=0, out=4096)
    a.update(kw)
    w = mx.mxrows_weight(*{**WEIGHT, **wkw}.values())
    a["weight"] = ctypes.byref(w) if a["weight"] else None
    assert mx.library().mxrows_product(*a.values(), None) == code


def test_product_workspace(mx):
    w = mx.mxrows_weight(*{**WEIGHT, "n": 4096, "k": 16384}.values())
    assert mx.mxrows_workspace_bytes(w, 4, 4) == 0 and mx.mxrows_workspace_bytes(w, 4, 65536) == 0
    need = mx.mxrows_workspace_bytes(w, 4, 203)
    assert 203 * 4096 * 4 * 2 <= need <= 16 << 20
    most = 0
    for rows in (33, 64, 65, 200, 256, 257, 1000, 5000):
        for n in (8, 64, 1000, 8192, 1 << 20):
            for k in (128, 2048, 65536):
                v = mx.mxrows_weight(*{**WEIGHT, "n": n, "k": k}.values())
                most = max(most, mx.mxrows_workspace_bytes(v, 4, rows))
    assert 0 < most <= 16 << 20
    lib = mx.library()
    for ws, nbytes, code in ((None, need, -4), (4096, need - 1, -4), (4104, need, -2)):
        assert lib.mxrows_product(ctypes.byref(w), 4, 4096, 4096, 203, ws, nbytes, 4096, None) == code
    for bad in (dict(experts=2), dict(n=12), dict(gated=3), dict(format=1)):
        assert mx.mxrows_workspace_bytes(mx.mxrows_weight(*{**WEIGHT, **bad}.values()), 4, 203) == 0
    assert mx.mxrows_workspace_bytes(w, 5, 203) == 0 and mx.mxrows_workspace_bytes(w, 4, 0) == 0


@pytest.mark.parametrize("wkw,kw,code", [(w, {}, c) for w, c in BAD_WEIGHTS] + [({}, kw, c) for kw, c in [
    (dict(weight=False), -1), (dict(f=0), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(out=None), -1),
    (dict(offsets=None), -1), (dict(rows=0), -1), (dict(x_rows=0), -1), (dict(gather=-1), -1), (dict(gather=33), -1), (dict(scatter=2), -1),
    (dict(order=None), -1), (dict(order=None, gather=0, scatter=1, x_rows=6), -1), (dict(gather=0), -1),
    (dict(x=4104), -2), (dict(out=4104), -2), (dict(offsets=4098), -2), (dict(order=4098), -2),
    (dict(f=8, x_rows=1 << 24), -5),  # 2^24 rows of 256 bytes: 4 GiB
]])
def test_grouped_refusals(mx, wkw, kw, code):
    a = dict(weight=True, f=4, x=4096, xs=4096, x_rows=3, order=4096, gather=2, scatter=0, offsets=4096, rows=6, out=4096)
    a.update(kw)
    w = mx.mxrows_weight(*{**WEIGHT, "experts": 3, **wkw}.values())
    a["weight"] = ctypes.byref(w) if a["weight"] else None
    assert mx.library().mxmoe_grouped(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), -1), (dict(order=None), -1), (dict(offsets=None), -1), (dict(tokens=0), -1), (dict(top_k=33), -1),
    (dict(experts=1025), -1), (dict(ids=4098), -2), (dict(order=4098), -2), (dict(offsets=4098), -2), (dict(ws=None), -4),
    (dict(nbytes=16), -4), (dict(ws=4104), -2),
])
def test_sort_refusals(mx, kw, code):
    a = dict(ids=4096, tokens=4000, top_k=2, experts=8, ws=4096, nbytes=1 << 20, order=4096, offsets=4096)
    a.update(kw)
    assert mx.library().mxmoe_sort(*a.values(), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), -1), (dict(ids=None), -1), (dict(weights=None), -1), (dict(out=None), -1), (dict(tokens=0), -1),
    (dict(top_k=0), -1), (dict(experts=0), -1), (dict(hidden=12), -1), (dict(hidden=0), -1),
    (dict(hidden=(1 << 20) + 8), -1), (dict(y=4104), -2), (dict(ids=4098), -2), (dict(weights=4098), -2),
    (dict(out=4104), -2),
])
def test_combine_refusals(mx, kw, code):
    a = dict(y=4096, ids=4096, weights=4096, tokens=4, top_k=2, experts=8, hidden=64, out=4096)
    a.update(kw)
    assert mx.library().mxmoe_combine(*a.values(), None) == code


def test_host_tensors_are_refused(mx):
    torch = pytest.importorskip("torch")
    from mxfp8_decode_gemm_amd import device as dv

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u = torch.zeros(4, 64, dtype=torch.uint8)
    for call in (lambda: dv.quantize4(x), lambda: dv.dequantize4(u, u), lambda: dv.quantize8(x), lambda: dv.Linear(u, u),
                 lambda: dv.GroupedLinear(u, u), lambda: dv.sort_pairs(u.int(), 4), lambda: dv.combine(x, u, x, 4)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
