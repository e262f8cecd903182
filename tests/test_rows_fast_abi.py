"""MXG_MXFP8_FAST without a GPU: a format of x alone, with the refusals of MXG_MXFP8."""

import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def mx():
    from mxfp8_decode_gemm_amd import build as b

    if not os.path.exists(b.LIB):
        b.build()
    from mxfp8_decode_gemm_amd import binding

    return binding


def _weight(mx, **kw):
    a = dict(w=4096, scale=4096, format=4, experts=1, n=4096, k=16384, gated=0)
    return mx.mxrows_weight(*{**a, **kw}.values())


def test_constant(mx):
    with open(mx.ROWS_HEADER_PATH) as f:
        line = [ln for ln in f if ln.startswith("#define MXG_MXFP8_FAST ")]
    assert len(line) == 1 and int(line[0].split()[2]) == mx.MXFP8_FAST == 9


def test_workspaces(mx):
    for form in (mx.MXFP4, mx.MXFP8):
        for x in (mx.MXFP8, mx.MXFP8_FAST):
            assert 0 < mx.mxrows_workspace_bytes(_weight(mx, format=form), x, 203) <= 16 << 20
            assert mx.mxrows_workspace_bytes(_weight(mx, format=form), x, 65536) == 0
    most = 0
    for rows in (33, 64, 65, 130, 200, 256, 257, 1000):
        for n in (8, 64, 1000, 8192):
            for k in (128, 2048, 65536):
                most = max(most, *(mx.mxrows_workspace_bytes(_weight(mx, format=8, n=n, k=k), x, rows) for x in (8, 9)))
    assert 0 < most <= 16 << 20


def test_no_format_of_weights(mx):
    assert mx.mxrows_packed_weight_bytes(mx.MXFP8_FAST, 1, 64, 256) == 0
    assert mx.mxrows_workspace_bytes(_weight(mx, format=mx.MXFP8_FAST), mx.MXFP8_FAST, 203) == 0


@pytest.mark.parametrize("kw,code", [(dict(x=None), -1), (dict(x=4104), -2), (dict(xs=4098), -2), (dict(out=None), -1),
                                     (dict(rows=0), -1), (dict(f=10), -1), (dict(ws=None), -4), (dict(nbytes=64), -4),
                                     (dict(ws=4104), -2)])
@pytest.mark.parametrize("form", [4, 8])
def test_refusals(mx, form, kw, code):
    a = dict(f=mx.MXFP8_FAST, x=4096, xs=4096, rows=203, ws=4096, nbytes=1 << 24, out=4096)
    a.update(kw)
    w = _weight(mx, format=form)
    assert mx.library().mxrows_product(ctypes.byref(w), *a.values(), None) == code


def test_gathered_rows_past_4_gib_are_refused(mx):
    w = _weight(mx, n=64, k=256)
    assert mx.library().mxmoe_grouped(ctypes.byref(w), mx.MXFP8_FAST, 4096, 4096, 1 << 24, 4096, 2, 0, 4096, 6, 4096,
                                      None) == -5
