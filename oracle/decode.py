"""The decode operators whose weights are chosen per row, in float64.

Test infrastructure only (see the package docstring). ``route``, ``experts``
and ``adapted`` restate the formulas of include/mxdecode.h one row at a time;
the last two also return how far a result computed in FP32 and rounded once to
BF16 may be off. The pieces of those bounds:

* a sum of K products in FP32, in any order: 1e-6 sum |products|, as in
  ``tolerance``;
* one BF16 rounding: one BF16 ulp of the exact value (half of it, doubled for
  a value that crosses a binade), as in ``tolerance``;
* h, or an adapter's u, held as two BF16 parts: the second part is at most 2^-9 |h| and rounded
  by 2^-9 of itself, so 2^-18 of the value;
* silu and its product in FP32: exp, add, divide and two multiplies at no more
  than 2 ulp (2^-23) each, so 10 * 2^-23 of |h|; a change of the gate by d
  moves silu by at most 1.1 d (the largest slope of silu is 1.0998).
"""

from __future__ import annotations

import numpy as np

from .codecs import bf16_quantum
from .gemm import dequantize
from .tolerance import REL_ABS_SUM

SILU_SLOPE = 1.1
H_ROUNDING = 2.0**-18 + 10 * 2.0**-23


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1,
          renormalize=False, scale=1.0):
    """(ids int32, weights float64) of [tokens, experts] logits."""
    logits = np.asarray(logits, dtype=np.float64)
    tokens, experts = logits.shape
    per = experts // groups
    ids = np.full((tokens, top_k), -1, dtype=np.int32)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens):
        row = logits[t]
        alive = [e for e in range(experts) if row[e] > -np.inf]  # not -infinity, not NaN
        if not alive:
            continue
        s = np.zeros(experts)
        if score == "softmax":
            top = max(row[e] for e in alive)
            for e in alive:
                s[e] = float(row[e] == top) if top == np.inf else np.exp(row[e] - top)
            s /= s.sum()
        else:
            for e in alive:
                s[e] = 1.0 / (1.0 + np.exp(-max(row[e], -709.0)))
        s[s < 2.0**-1022] = 0.0  # below FP64's normal range
        c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        if groups > 1:
            best = []
            for g in range(groups):
                mine = sorted((c[e] for e in alive if e // per == g), reverse=True)
                if mine:
                    best.append((-sum(mine[:group_best]), g))
            kept = {g for _, g in sorted(best)[:top_groups]}
            alive = [e for e in alive if e // per in kept]
        chosen = sorted(alive, key=lambda e: (-c[e], e))[:top_k]
        w = np.array([s[e] for e in chosen])
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, : len(chosen)] = chosen
        weights[t, : len(chosen)] = w * scale
    return ids, weights


def _bf16_weight(codes, scales):
    """MXFP8 weights as the BF16 values nearest to code times scale (the value
    itself for scale bytes 3..246)."""
    v = dequantize(codes, scales)
    step = bf16_quantum(v)
    return np.rint(v / step) * step


def experts(x, ids, weights, w13, w13_scale, w2, w2_scale):
    """(exact, bound) [tokens, hidden] of float64 x and MXFP8 experts."""
    x = np.asarray(x, dtype=np.float64)
    count, _, inter = w2.shape
    exact, slack, mass = (np.zeros_like(x) for _ in range(3))
    cache = {}
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < count:
                continue
            if e not in cache:
                cache[e] = (_bf16_weight(w13[e], w13_scale[e]), _bf16_weight(w2[e], w2_scale[e]))
            up, down = cache[e]
            z, za = up @ x[t], REL_ABS_SUM * (np.abs(up) @ np.abs(x[t]))
            g, u = z[:inter], z[inter:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            dh = SILU_SLOPE * za[:inter] * (np.abs(u) + za[inter:]) + np.abs(silu) * za[inter:]
            dh = dh + H_ROUNDING * np.abs(h)
            y, ya = down @ h, np.abs(down) @ (np.abs(h) + dh)
            w = float(weights[t, j])
            exact[t] += w * y
            slack[t] += abs(w) * (np.abs(down) @ dh + REL_ABS_SUM * ya)
            mass[t] += abs(w) * np.abs(y)
    return exact, bf16_quantum(exact) + slack + REL_ABS_SUM * mass


def adapted(x_shared, x, w, w_scale, a, b, scale, ids):
    """(exact, bound) [m, n]: float64 x of the shared product (quantized) and
    of the adapters, MXFP8 w, float64 a [adapters, rank, k], b [adapters, n,
    rank]."""
    wv = dequantize(w, w_scale)
    exact = x_shared @ wv.T
    slack = REL_ABS_SUM * (np.abs(x_shared) @ np.abs(wv).T)
    for t, i in enumerate(ids):
        if not 0 <= i < len(a):
            continue
        u = a[i] @ x[t]
        du = REL_ABS_SUM * (np.abs(a[i]) @ np.abs(x[t])) + (2.0**-18 + 2.0**-23) * np.abs(u)
        exact[t] += scale[i] * (b[i] @ u)
        slack[t] += abs(scale[i]) * (np.abs(b[i]) @ (du + REL_ABS_SUM * np.abs(u)))
    return exact, bf16_quantum(exact) + slack + 2.0**-23 * np.abs(exact)
