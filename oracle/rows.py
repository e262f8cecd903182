"""The products of any number of rows in MXFP4 and MXFP8, in float64.

Test infrastructure only (see the package docstring). Restates include/mxrows.h: the MXFP4 quantizer, the
products (dense, gated, grouped by expert), the sort of a router's pairs and their weighted sum. The products also
return how far a result may be off before its rounding to BF16; ``bf16_bound`` adds that rounding. The pieces:

* an FP32 sum of K products, taken eight at a time: at most K/8 additions, and 16 more where partial sums of
  waves meet, each off by no more than 2^-23 of the sum of magnitudes;
* with MXFP8 rows that are to be fast, or that BF16 does not hold with their scales (a scale byte outside 3..246 beside
  a nonzero code, in W or x), the matrix instruction drops, of eight products at aligned K, what lies below 2^-13 of the
  largest: at most 7 * 2^-13 of it. The largest magnitudes of the eight of W and of x bound that product;
* silu and its product in FP32: (10 + |gate|) * 2^-23 of the result (the exponential as three factors of 1 ulp each, a
  reciprocal of 1 ulp, eight products and sums of half a step: 8 * 2^-23; the exponent -|gate| log2(e), rounded to 2^-24
  of itself by its product and by its constant, moves exp by |gate| 2^-23 of it at most); a change of the gate by d moves
  silu by at most 1.1 d;
* one BF16 rounding: half a step, at most 2^-8 of the value.
"""

from __future__ import annotations

import math

import numpy as np

from .codecs import decode_e4m3, decode_e8m0
from .quant import BLOCK

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SILU_SLOPE = 1.1
GATE_ROUNDING = 2.0**-23


def e2m1_value(code: int) -> float:
    """The value of a 4-bit code, from its fields: sign, two exponent bits (bias 1), one mantissa bit."""
    sign = -1.0 if code & 8 else 1.0
    exp, man = (code >> 1) & 3, code & 1
    return sign * (man * 0.5 if exp == 0 else (1 + man / 2) * 2.0 ** (exp - 1))


def e2m1_round(y: float) -> int:
    """The code of the E2M1 value nearest to y, |y| <= 6, ties to the even code, the sign kept."""
    if math.isnan(y) or abs(y) > 6:
        raise ValueError("value outside the E2M1 range")
    a = abs(y)
    best = min(range(8), key=lambda c: (abs(E2M1[c] - a), c & 1))
    return best | (8 if math.copysign(1.0, y) < 0 else 0)


def fp4_exponent(amax: float) -> int:
    """Smallest integer e with amax <= 6 * 2^e, clamped to [-127, 127]; -127 for zero."""
    if amax == 0.0:
        return -127
    e = math.frexp(amax)[1] - 3
    while 6 * math.ldexp(1.0, e) < amax:
        e += 1
    while 6 * math.ldexp(1.0, e - 1) >= amax:
        e -= 1
    return max(-127, min(127, e))


def pack4(codes: np.ndarray) -> np.ndarray:
    """Two codes a byte, the lower index in the low half."""
    codes = np.asarray(codes, dtype=np.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack4(b: np.ndarray) -> np.ndarray:
    b = np.asarray(b, dtype=np.uint8)
    return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def quantize4(values: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(packed codes, scale bytes) of [rows, K] float values, element by element."""
    values = np.asarray(values, dtype=np.float64)
    rows, k = values.shape
    codes = np.zeros((rows, k), dtype=np.uint8)
    scales = np.zeros((rows, k // BLOCK), dtype=np.uint8)
    for r in range(rows):
        for b in range(k // BLOCK):
            block = [float(v) for v in values[r, b * BLOCK : (b + 1) * BLOCK]]
            if all(math.isfinite(v) for v in block):
                e = fp4_exponent(max(abs(v) for v in block))
                scales[r, b] = e + 127
                found = [e2m1_round(math.ldexp(v, -e)) for v in block]
            else:
                scales[r, b] = 0xFF
                found = [7 | (8 if math.copysign(1.0, v) < 0 else 0) for v in block]
            codes[r, b * BLOCK : (b + 1) * BLOCK] = found
    return pack4(codes), scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of codes (MXFP4 where there are 16 bytes for each scale byte, else MXFP8) and scale bytes; NaN
    where the scale byte is 255."""
    scales = np.asarray(scales, dtype=np.uint8)
    if codes.shape[-1] == 16 * scales.shape[-1]:
        v = np.array([e2m1_value(c) for c in range(16)])[unpack4(codes)]
    else:
        v = decode_e4m3(np.asarray(codes, dtype=np.uint8))
    factor = np.where(scales == 0xFF, np.nan, decode_e8m0(np.where(scales == 0xFF, 0, scales)))
    return v * np.repeat(factor, BLOCK, axis=-1)


def is_mxfp8(codes: np.ndarray, scales: np.ndarray) -> bool:
    return codes.shape[-1] == 32 * scales.shape[-1]


def leaves_bf16(v, scales):
    """Whether values, given with their scale bytes, hold a nonzero one whose scale byte is outside 3..246."""
    outside = np.repeat((scales < 3) | (scales > 246), BLOCK, axis=-1)
    return bool((outside & (v != 0)).any())


def product(w, w_scale, x, x_scale, gated=False, fast=False):
    """(exact, slack) [rows, n]: W x of every row; gated: silu(gate) * up, [rows, n/2]."""
    wv, xv = values(w, w_scale), values(x, x_scale)
    k = wv.shape[1]
    exact = xv @ wv.T
    slack = (k / 8 + 16) * 2.0**-23 * (np.abs(xv) @ np.abs(wv).T)
    if is_mxfp8(x, x_scale) and (fast or leaves_bf16(wv, w_scale) or leaves_bf16(xv, x_scale)):
        largest = lambda v: np.abs(v).reshape(len(v), -1, 8).max(-1)  # noqa: E731
        slack += 7 * 2.0**-13 * (largest(xv) @ largest(wv).T)
    if not gated:
        return exact, slack
    half = wv.shape[0] // 2
    g, u, dg, du = exact[:, :half], exact[:, half:], slack[:, :half], slack[:, half:]
    silu = g / (1 + np.exp(-g))
    h = silu * u
    return h, SILU_SLOPE * dg * (np.abs(u) + du) + np.abs(silu) * du + GATE_ROUNDING * (10 + np.abs(g)) * np.abs(h)


def sort_pairs(ids, experts):
    """(order, offsets): the flat pairs by expert, an expert's in ascending order, those without one last."""
    ids = [int(e) for e in np.asarray(ids).ravel()]
    order, offsets = [], [0]
    for e in range(experts):
        order += [p for p, i in enumerate(ids) if i == e]
        offsets.append(len(order))
    order += [p for p, i in enumerate(ids) if not 0 <= i < experts]
    return np.array(order, dtype=np.int32), np.array(offsets, dtype=np.int32)


def grouped(w, w_scale, x, x_scale, offsets, order=None, gather=0, scatter=False, gated=False, rows=None,
            fast=False):
    """(exact, slack, written) [rows, ...]; written: which rows the experts' pairs lead to."""
    rows = len(x) if rows is None else rows
    width = w.shape[1] // 2 if gated else w.shape[1]
    exact, slack = np.zeros((rows, width)), np.zeros((rows, width))
    written = np.zeros(rows, dtype=bool)
    for e in range(len(w)):
        at = np.arange(offsets[e], offsets[e + 1])
        if not len(at):
            continue
        src = order[at] // gather if gather else at
        dst = order[at] if scatter else at
        exact[dst], slack[dst] = product(w[e], w_scale[e], x[src], x_scale[src], gated, fast)
        written[dst] = True
    return exact, slack, written


def combine(y, ids, weights, experts):
    """(exact, slack) [tokens, hidden] of float64 y [tokens, top_k, hidden]."""
    there = (ids >= 0) & (ids < experts)
    p = np.where(there[..., None], y, 0.0) * np.where(there, weights, 0.0)[..., None].astype(np.float64)
    return p.sum(1), ids.shape[1] * 2.0**-23 * np.abs(p).sum(1)


def bf16_bound(exact, slack):
    """How far a BF16 result may be from the exact value."""
    return slack + 2.0**-8 * (np.abs(exact) + slack) + 2.0**-134
