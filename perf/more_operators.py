"""Workloads of the products of any number of rows in MXFP4 and MXFP8, with their plain forms.

Five operators, each in its plain form (elementary torch operations in 32 bits) and as the library's call:

* quantize: rows to MXFP4 and back: per 32 values the smallest e with amax <= 6 2^e, E2M1 codes nearest to v / 2^e (ties to
  even), then the values that codes and scales stand for, in BF16 (exact).
* linear: C[t, n] = sum_k W[n, k] x[t, k] for any number of rows; W and x in MXFP4 or MXFP8. Gated, with W = [Wg; Wu]:
  silu(Wg x) * (Wu x).
* sort: the (token, choice) pairs of a router, stably by expert: order, and where each expert's pairs begin. Pairs
  without an expert come last.
* grouped: the same product, each expert's weight on the rows of its pairs. gather: row i of the sorted ones is x[order[i] //
  top_k]; scatter: its result is row order[i].
* combine: out[t] = sum_j weights[t, j] y[t, j] over the choices that are experts.

MXFP4 is E2M1 codes (two a byte, the lower index in the low half) with one E8M0 scale byte per 32 values along the last
dimension, MXFP8 e4m3fn codes with the same scales.
"""

from __future__ import annotations

import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # The activations of one decode step: latency.
        dict(name="quantize 8x7168 bf16", op="quantize", rows=8, k=7168, pad=0, dtype="bfloat16"),
        # A prefill of 16384 tokens: bandwidth.
        dict(name="quantize 16384x8192 bf16", op="quantize", rows=16384, k=8192, pad=0, dtype="bfloat16"),
        # One token through the headline projection with 4-bit weights: the weight stream.
        dict(name="linear 1 7168x8192 w4x4", op="linear", rows=1, n=7168, k=8192, w="mxfp4", x="mxfp4", gated=False),
        # A prompt through the same projection: matrix cores.
        dict(name="linear 4096 7168x8192 w4x4", op="linear", rows=4096, n=7168, k=8192, w="mxfp4", x="mxfp4", gated=False),
        # A ragged batch of drafted tokens through a long K: 4-bit weights on 8-bit activations.
        dict(name="linear 203 4096x16384 w4x8", op="linear", rows=203, n=4096, k=16384, w="mxfp4", x="mxfp8", gated=False),
        # The pairs of a decode step: latency.
        dict(name="sort 8x8 of 64", op="sort", tokens=8, top_k=8, experts=64, dropped=0.0),
        # The pairs of a prefill over many experts, some tokens without all their choices.
        dict(name="sort 16384x8 of 256", op="sort", tokens=16384, top_k=8, experts=256, dropped=0.02),
        # The gated product of one decode step: few rows for each of about 42 experts, the weight stream.
        dict(name="grouped 8x8 of 64 4096x7168 w4x8 gated", op="grouped", tokens=8, top_k=8, experts=64, n=4096, k=7168,
             w="mxfp4", x="mxfp8", gated=True, form="gather"),
        # The same over a prompt: matrix cores, experts of very different popularity.
        dict(name="grouped 4096x8 of 64 4096x7168 w4x4 gated", op="grouped", tokens=4096, top_k=8, experts=64, n=4096,
             k=7168, w="mxfp4", x="mxfp4", gated=True, form="gather"),
        # The product back to the hidden size with 8-bit weights, an odd number of tokens, results in the pairs' own order.
        dict(name="grouped 1001x2 of 8 4096x1024 w8x8", op="grouped", tokens=1001, top_k=2, experts=8, n=4096, k=1024,
             w="mxfp8", x="mxfp8", gated=False, form="scatter"),
        # A decode step's weighted sum: latency.
        dict(name="combine 8x8x7168", op="combine", tokens=8, top_k=8, experts=64, hidden=7168, dropped=0.0),
        # A prompt's: bandwidth.
        dict(name="combine 4096x8x7168", op="combine", tokens=4096, top_k=8, experts=64, hidden=7168, dropped=0.02),
    ]


_FORMATS = [("mxfp4", "mxfp4"), ("mxfp4", "mxfp8"), ("mxfp8", "mxfp8")]  # of W and x


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "sort", "grouped", "grouped", "combine"])
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 16384), k=32 * _log_int(rng, 1, 256), pad=rng.choice([0, 0, 8, 96]),
                    dtype=rng.choice(["bfloat16", "float16", "float32"]))
    if op == "sort":
        experts = _log_int(rng, 2, 512)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), top_k=rng.randint(1, min(8, experts)), experts=experts,
                    dropped=rng.choice([0.0, 0.02, 0.5]))
    if op == "combine":
        experts = rng.randint(2, 256)
        return dict(op=op, tokens=_log_int(rng, 1, 4096), top_k=rng.randint(1, min(8, experts)), experts=experts,
                    hidden=128 * _log_int(rng, 1, 56), dropped=rng.choice([0.0, 0.02, 0.5]))
    w, x = rng.choice(_FORMATS)
    gated = rng.random() < 0.4
    n = 64 * _log_int(rng, 1, 112) if gated else 8 * _log_int(rng, 4, 896)
    k = 128 * _log_int(rng, 1, 64)
    if op == "linear":
        return dict(op=op, rows=_log_int(rng, 1, 4096), n=n, k=k, w=w, x=x, gated=gated)
    while True:
        experts, tokens = rng.randint(2, 64), _log_int(rng, 1, 4096)
        top_k = rng.randint(1, min(8, experts))
        # no more weights, and no more rows times weights, than the largest listed case
        if experts * n * k <= 64 * 4096 * 7168 and tokens * top_k * n * k <= 4096 * 8 * 4096 * 7168:
            return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, n=n, k=k, w=w, x=x, gated=gated,
                        form=rng.choice(["gather", "scatter", "plain"]))


_BYTES = {"mxfp4": 17 / 32, "mxfp8": 33 / 32}  # of one value


def work(case):
    if case["op"] == "quantize":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": int(case["rows"] * case["k"] * (size + 2 * _BYTES["mxfp4"] + 2)), "flops": 0}
    if case["op"] == "sort":
        return {"bytes": 8 * case["tokens"] * case["top_k"] + 4 * case["experts"] + 4, "flops": 0}
    if case["op"] == "combine":
        pairs = case["tokens"] * case["top_k"]
        kept = int(pairs * (1 - case["dropped"]))
        return {"bytes": 2 * case["hidden"] * (kept + case["tokens"]) + 8 * pairs, "flops": 2 * kept * case["hidden"]}
    n, k = case["n"], case["k"]
    out = n // 2 if case["gated"] else n
    if case["op"] == "linear":
        rows, x_rows, active = case["rows"], case["rows"], 1
    else:
        t, e, c = case["tokens"], case["experts"], case["top_k"]
        rows, x_rows = t * c, t if case["form"] == "gather" else t * c
        active = e * (1.0 - (1.0 - c / e) ** t)  # distinct experts of t independent choices of c
    return {"bytes": int(active * n * k * _BYTES[case["w"]] + x_rows * k * _BYTES[case["x"]] + 2 * rows * out),
            "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _encode4(v):
    """MXFP4 codes (two a byte) and scale bytes of finite values, in the type that they come in."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    f, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(f > 0.75, p - 2, p - 3)
    e = torch.where(f == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    y = torch.ldexp(b, -e.unsqueeze(-1)).reshape(v.shape)
    a = y.abs()
    code = (a > 0.25).byte()  # ties go to the even code
    for border, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= border) if even else (a > border)
    code |= torch.signbit(y).byte() << 3
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).byte()


def _encode8(v):
    """MXFP8 codes and scale bytes of finite float32 values: per 32, the smallest e with amax <= 448 2^e."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    f, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(f > 0.875, p - 8, p - 9)
    e = torch.where(f == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(v.shape), (e + 127).byte()


_ENCODE = {"mxfp4": _encode4, "mxfp8": _encode8}


def _weights(gen, form, experts, n, k):
    """Weights of standard deviation 1/sqrt(K), one matrix at a time."""
    codes = torch.empty(experts, n, k // 2 if form == "mxfp4" else k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(experts, n, k // 32, dtype=torch.uint8, device="cuda")
    for i in range(experts):
        c, s = _ENCODE[form](torch.randn(n, k, generator=gen, device="cuda") * k**-0.5)
        codes[i].copy_(c)
        scales[i].copy_(s)
    return codes, scales


def _rows(gen, rows, k):
    """Activations: Gaussians with 1 % of the channels ten times as large."""
    x = torch.randn(rows, k, generator=gen, device="cuda")
    x[:, torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 100)]] *= 10
    return x


def _choices(gen, tokens, experts, top_k, dropped=0.0):
    """A router's choices: distinct experts of a token, some experts several times as popular as others."""
    noise = torch.rand(tokens, experts, generator=gen, device="cuda").clamp(1e-6, 1 - 1e-6)
    liked = 0.7 * torch.randn(experts, generator=gen, device="cuda")
    ids = (liked - torch.log(-torch.log(noise))).topk(top_k).indices.int()
    lost = torch.rand(tokens, top_k, generator=gen, device="cuda") < dropped
    return torch.where(lost, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        x = _rows(gen, case["rows"], case["k"] + case["pad"]).to(getattr(torch, case["dtype"]))
        s["x"] = x[:, : case["k"]]
    elif case["op"] == "sort":
        s["ids"] = _choices(gen, case["tokens"], case["experts"], case["top_k"], case["dropped"])
    elif case["op"] == "combine":
        t, j = case["tokens"], case["top_k"]
        s["ids"] = _choices(gen, t, case["experts"], j, case["dropped"])
        s["weights"] = torch.softmax(torch.randn(t, j, generator=gen, device="cuda"), -1)
        s["y"] = torch.randn(t * j, case["hidden"], generator=gen, device="cuda").bfloat16()
    elif case["op"] == "linear":
        s["w"], s["w_scale"] = (v[0] for v in _weights(gen, case["w"], 1, case["n"], case["k"]))
        s["x"], s["x_scale"] = _ENCODE[case["x"]](_rows(gen, case["rows"], case["k"]))
        if own:  # the weight laid out once, as a server keeps it
            from mxfp8_decode_gemm_amd import device as dv

            s["handle"] = dv.Linear(s["w"], s["w_scale"], gated=case["gated"])
    else:
        t, e, j = case["tokens"], case["experts"], case["top_k"]
        s["w"], s["w_scale"] = _weights(gen, case["w"], e, case["n"], case["k"])
        rows = t if case["form"] == "gather" else t * j
        s["x"], s["x_scale"] = _ENCODE[case["x"]](_rows(gen, rows, case["k"]))
        ids = _choices(gen, t, e, j).flatten().long()
        s["order"] = ids.argsort(stable=True).int()
        count = torch.bincount(ids, minlength=e)
        s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
        s["most"] = int(count.max())  # rows of the most popular expert
        if own:
            from mxfp8_decode_gemm_amd import device as dv

            s["handle"] = dv.GroupedLinear(s["w"], s["w_scale"], gated=case["gated"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _library(s)
    return {"quantize": _quantize, "linear": _linear, "sort": _sort, "grouped": _grouped, "combine": _combine}[s["op"]](s)


def _library(s):
    from mxfp8_decode_gemm_amd import device as dv

    if s["op"] == "quantize":
        return dv.dequantize4(*dv.quantize4(s["x"]), dtype=torch.bfloat16)
    if s["op"] == "sort":
        return dv.sort_pairs(s["ids"], s["experts"])
    if s["op"] == "combine":
        return dv.combine(s["y"], s["ids"], s["weights"], s["experts"])
    if s["op"] == "linear":
        return s["handle"](s["x"], s["x_scale"])
    return s["handle"](s["x"], s["x_scale"], s["offsets"], order=None if s["form"] == "plain" else s["order"],
                       gather=s["top_k"] if s["form"] == "gather" else 0, scatter=s["form"] == "scatter")


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _decode(codes, scales):
    """The float32 values of codes and scale bytes (1..254: a scale byte is the exponent field of its value); MXFP4 codes
    are half as many bytes."""
    if codes.shape[-1] == 16 * scales.shape[-1]:
        table = torch.tensor(_E2M1, device=codes.device)
        both = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)  # of a byte
        v = both[codes.int()].flatten(-2)
    else:
        v = codes.view(torch.float8_e4m3fn).float()
    step = (scales.int() << 23).view(torch.float32)
    return (v.view(*v.shape[:-1], -1, 32) * step.unsqueeze(-1)).view(v.shape)


def _gate(z):
    gate, up = z.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _quantize(s):
    return _decode(*_encode4(s["x"].float())).bfloat16()


def _linear(s):
    z = _decode(s["x"], s["x_scale"]) @ _decode(s["w"], s["w_scale"]).t()
    return (_gate(z) if s["gated"] else z).bfloat16()


def _sort(s):
    ids, experts = s["ids"].flatten().long(), s["experts"]
    key = torch.where((ids < 0) | (ids >= experts), torch.full_like(ids, experts), ids)
    order = key.argsort(stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=key.device))
    return order.int(), offsets.int()


def _grouped(s):
    """Every expert's rows in a matrix of its own, as long as the longest."""
    x, order, offsets = _decode(s["x"], s["x_scale"]), s["order"].long(), s["offsets"].long()
    i = torch.arange(order.shape[0], device=x.device)
    e = torch.searchsorted(offsets, i, right=True) - 1
    at = i - offsets[e]
    rows = x.new_zeros(s["experts"], s["most"], s["k"])
    rows[e, at] = x[order // s["top_k"]] if s["form"] == "gather" else x
    z = (rows @ _decode(s["w"], s["w_scale"]).transpose(1, 2).contiguous())[e, at]
    z = (_gate(z) if s["gated"] else z).bfloat16()
    return torch.empty_like(z).index_copy_(0, order, z) if s["form"] == "scatter" else z


def _combine(s):
    t, j = s["ids"].shape
    there = (s["ids"] >= 0) & (s["ids"] < s["experts"])
    w = torch.where(there, s["weights"], torch.zeros_like(s["weights"]))
    return (s["y"].float().view(t, j, -1) * w.unsqueeze(-1)).sum(1).bfloat16()


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _value64(codes, scales):
    """float64 values from the bits: sign, 2 or 4 exponent bits (bias 1 or 7), 1 or 3 mantissa bits; scale byte s is
    2^(s - 127)."""
    c = codes.long()
    if codes.shape[-1] == 16 * scales.shape[-1]:
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        sign, ex, mant, bias, half = c >> 3, (c >> 1) & 3, (c & 1).double() / 2, 1, 2.0
    else:
        sign, ex, mant, bias, half = c >> 7, (c >> 3) & 15, (c & 7).double() / 8, 7, 2.0**-5
    mag = torch.where(ex == 0, mant * (half / 2), torch.ldexp(1 + mant, ex - bias))
    v = torch.where(sign == 1, -mag, mag)
    return torch.ldexp(v, scales.long().repeat_interleave(32, -1) - 127)


def _silu64(z):
    half = z.shape[-1] // 2
    return z[..., :half] * torch.sigmoid(z[..., :half]) * z[..., half:]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        b = s["x"].double().reshape(case["rows"], -1, 32)
        amax = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(amax.clamp_min(2.0**-126) / 6)) - 1
        for _ in range(3):
            e = torch.where(6 * torch.exp2(e) < amax, e + 1, e)
        y = b / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(1.0))).clamp_min(0) - 1)
        return (torch.round(y / step) * step * torch.exp2(e)).reshape(case["rows"], -1)
    if case["op"] == "sort":
        ids, experts = s["ids"].flatten().cpu(), case["experts"]
        groups = [(ids == e).nonzero().flatten() for e in range(experts)]
        order = torch.cat(groups + [((ids < 0) | (ids >= experts)).nonzero().flatten()])
        ends = torch.tensor([0] + [g.numel() for g in groups]).cumsum(0)
        return order.int(), ends.int()
    if case["op"] == "combine":
        t, j = case["tokens"], case["top_k"]
        out = torch.zeros(t, case["hidden"], dtype=torch.float64, device="cuda")
        y = s["y"].view(t, j, -1)
        for c in range(j):
            w = s["weights"][:, c].double() * ((s["ids"][:, c] >= 0) & (s["ids"][:, c] < case["experts"]))
            out += w.unsqueeze(-1) * y[:, c].double()
        return out
    x = _value64(s["x"], s["x_scale"])
    if case["op"] == "linear":
        z = x @ _value64(s["w"], s["w_scale"]).t()
        return _silu64(z) if case["gated"] else z
    order, ends = s["order"].long(), s["offsets"].tolist()
    out = torch.zeros(order.shape[0], case["n"] // 2 if case["gated"] else case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        i = torch.arange(ends[e], ends[e + 1], device="cuda")
        if i.numel():
            z = x[order[i] // case["top_k"] if case["form"] == "gather" else i] @ _value64(s["w"][e], s["w_scale"][e]).t()
            out[order[i] if case["form"] == "scatter" else i] = _silu64(z) if case["gated"] else z
    return out
