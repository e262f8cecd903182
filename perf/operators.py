"""Workloads of the decode operators whose weights are chosen per row, with their plain forms.

Three operators, each in its plain form (elementary torch operations in 32 bits, 64 where a border decides)
and as the library's call:

* route: expert scores (softmax or sigmoid) of a row of logits, a bias that counts for the choice only, group
  limited top-k, the chosen scores as weights, renormalised when asked.
* experts: the gated MXFP8 products of the chosen experts, out[t] = sum_j weight[t, j] W2[e] (silu(Wg[e] x) * Wu[e] x)
  with e = ids[t, j], W13 = [Wg; Wu].
* adapted: the MXFP8 projection of at most 8 rows with each row's low-rank adapter beside it,
  out[t] = W q(x)[t] + scale[a] B[a] (A[a] x[t]) with a = ids[t] (none below 0). BF16 x is quantized for the shared
  product (one E8M0 scale per 32), the adapter takes it as it is.

MXFP8 here is e4m3fn codes with one E8M0 scale byte per 32 values along the last dimension.
"""

from __future__ import annotations

import numpy as np
import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

# A decode step has at most 8 rows (the library's GEMM limit); 64 rows are eight such steps or a batch of drafted tokens.
# Prefill reaches the router alone, with the longest sequence the sizes here name (16384).


def listed():
    return [
        # The router of one decode step: grouped sigmoid choice with a balance bias. Latency is what counts.
        dict(name="route 8x256 sigmoid groups", op="route", tokens=8, experts=256, top_k=8, score="sigmoid", groups=8,
             top_groups=4, group_best=2, bias=True, renormalize=True, scale=2.5, dtype="float32"),
        # The same router over a prefill of 16384 tokens: bandwidth and selection work.
        dict(name="route 16384x256 sigmoid groups", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid",
             groups=8, top_groups=4, group_best=2, bias=True, renormalize=True, scale=2.5, dtype="float32"),
        # BF16 logits (as the library's GEMM writes them), softmax, an odd number of tokens and experts, no groups.
        dict(name="route 1001x60 softmax", op="route", tokens=1001, experts=60, top_k=4, score="softmax", groups=1,
             top_groups=1, group_best=1, bias=False, renormalize=False, scale=1.0, dtype="bfloat16"),
        # One token through 8 of 64 experts of the headline width: the weight stream of the smallest decode step.
        dict(name="experts t1 7168x2048 8of64", op="experts", tokens=1, experts=64, top_k=8, hidden=7168, inter=2048),
        # A full decode step: 8 tokens, about 42 experts' weights.
        dict(name="experts t8 7168x2048 8of64", op="experts", tokens=8, experts=64, top_k=8, hidden=7168, inter=2048),
        # Many rows per expert: 64 drafted tokens over few experts.
        dict(name="experts t64 4096x1024 2of8", op="experts", tokens=64, experts=8, top_k=2, hidden=4096, inter=1024),
        # A small ragged one: sizes that are no power of two, 3 tokens. Latency is what counts.
        dict(name="experts t3 896x384 2of8", op="experts", tokens=3, experts=8, top_k=2, hidden=896, inter=384),
        # The headline projection with every row on its own rank-16 adapter.
        dict(name="adapted 8 7168x8192 s4 r16", op="adapted", rows=8, n=7168, k=8192, split_k=4, rank=16, adapters=32,
             used=8, bare=0, x="bf16"),
        # Four rows on two adapters of a large rank, no split.
        dict(name="adapted 4 7168x2048 s1 r64", op="adapted", rows=4, n=7168, k=2048, split_k=1, rank=64, adapters=8,
             used=2, bare=0, x="bf16"),
        # A long K with quantized x, rows without an adapter among the others.
        dict(name="adapted 5 4096x16384 s8 r32", op="adapted", rows=5, n=4096, k=16384, split_k=8, rank=32, adapters=16,
             used=3, bare=2, x="mxfp8"),
        # The tiny projection: one row, launch latency.
        dict(name="adapted 1 256x512 s1 r8", op="adapted", rows=1, n=256, k=512, split_k=1, rank=8, adapters=4, used=1,
             bare=0, x="bf16"),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "experts", "adapted"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, 8, 512) // groups
        per = max(per, 2)
        experts = per * groups
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, per * top_groups))
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, top_k=top_k,
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups, top_groups=top_groups,
                    group_best=rng.choice([1, 2]), bias=rng.random() < 0.5, renormalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["float32", "bfloat16"]))
    if op == "experts":
        while True:
            tokens, experts = _log_int(rng, 1, 64), rng.randint(4, 64)
            top_k = rng.randint(1, min(8, experts))
            hidden, inter = 128 * _log_int(rng, 1, 56), 128 * _log_int(rng, 1, 16)
            # no more weights, and no more rows times weights, than the largest listed case
            if experts * hidden * inter <= 64 * 7168 * 2048 and tokens * top_k * hidden * inter <= 64 * 7168 * 2048:
                return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, hidden=hidden, inter=inter)
    split_k = rng.choice([1, 2, 4, 8])
    rows, adapters = rng.randint(1, 8), rng.randint(1, 32)
    bare = rng.choice([0, 0, rng.randint(0, rows)])
    return dict(op=op, rows=rows, n=8 * _log_int(rng, 8, 512 if split_k == 8 else 1024),
                k=128 * split_k * _log_int(rng, 1, 128 // split_k), split_k=split_k, rank=8 * _log_int(rng, 1, 16),
                adapters=adapters, used=min(rows - bare, rng.randint(1, adapters)), bare=bare,
                x=rng.choice(["bf16", "mxfp8"]))


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 8 * t * k, "flops": 4 * t * e}
    if case["op"] == "experts":
        t, e, k, h, i = (case[n] for n in ("tokens", "experts", "top_k", "hidden", "inter"))
        active = e * (1.0 - (1.0 - k / e) ** t)  # distinct experts of t independent choices of k
        return {"bytes": int(active * 3 * h * i * 33 / 32) + 4 * t * h + 8 * t * k, "flops": 6 * t * k * h * i}
    m, n, k, r = (case[x] for x in ("rows", "n", "k", "rank"))
    x = 2 * m * k if case["x"] == "bf16" else m * k * 33 // 32
    return {"bytes": n * k * 33 // 32 + x + 2 * case["used"] * r * (n + k) + 2 * m * n,
            "flops": 2 * m * n * k + 2 * (m - case["bare"]) * r * (n + k)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _encode(v):
    """MXFP8 codes and scale bytes of finite float32 values: per 32, the smallest e with amax <= 448 2^e."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    f, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(f > 0.875, p - 8, p - 9)
    e = torch.where(f == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    codes = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(v.shape), (e + 127).to(torch.uint8)


def _weights(gen, *shape):
    """MXFP8 weights of standard deviation 1/sqrt(K), one matrix at a time."""
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty(*shape[:-1], shape[-1] // 32, dtype=torch.uint8, device="cuda")
    for i in range(shape[0] if len(shape) == 3 else 1):
        c, s = (codes[i], scales[i]) if len(shape) == 3 else (codes, scales)
        q, e = _encode(torch.randn(shape[-2:], generator=gen, device="cuda") * shape[-1] ** -0.5)
        c.copy_(q)
        s.copy_(e)
    return codes, scales


def _rows(gen, rows, k):
    """BF16 activations: Gaussians with 1 % of the channels ten times as large."""
    x = torch.randn(rows, k, generator=gen, device="cuda")
    x[:, torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 100)]] *= 10
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        s["logits"] = (1.5 * torch.randn(t, e, generator=gen, device="cuda")).to(getattr(torch, case["dtype"]))
        s["bias"] = 0.1 * torch.randn(e, generator=gen, device="cuda") if case["bias"] else None
    elif case["op"] == "experts":
        t, e, k, h, i = (case[n] for n in ("tokens", "experts", "top_k", "hidden", "inter"))
        s["w13"], s["w13_scale"] = _weights(gen, e, 2 * i, h)
        s["w2"], s["w2_scale"] = _weights(gen, e, h, i)
        s["x"] = _rows(gen, t, h)
        top = torch.rand(t, e, generator=gen, device="cuda").topk(k)
        s["ids"], s["weights"] = top.indices.int(), top.values / top.values.sum(-1, keepdim=True)
        if own:  # the weights in the streaming layout and the workspace, as a server keeps them
            from mxfp8_decode_gemm_amd import device as dv

            s["handle"] = dv.Experts(s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], t * k)
    else:
        m, n, k, r, count = (case[x] for x in ("rows", "n", "k", "rank", "adapters"))
        s["w"], s["w_scale"] = _weights(gen, n, k)
        s["x"], s["x_scale"] = _rows(gen, m, k), None
        if case["x"] == "mxfp8":
            s["x"], s["x_scale"] = _encode(s["x"].float())
        s["a"] = (torch.randn(count, r, k, generator=gen, device="cuda") * k**-0.5).bfloat16()
        s["b"] = (torch.randn(count, n, r, generator=gen, device="cuda") * r**-0.5).bfloat16()
        s["scale"] = 0.5 + torch.rand(count, generator=gen, device="cuda")
        chosen = torch.randperm(count, generator=gen, device="cuda")[: max(1, case["used"])]
        ids = chosen[torch.arange(m, device="cuda") % chosen.numel()]
        ids[: case["bare"]] = -1
        s["ids"] = ids[torch.randperm(m, generator=gen, device="cuda")].int()
        if own:
            from mxfp8_decode_gemm_amd import device as dv

            s["handle"] = dv.AdaptedLinear(s["w"], s["w_scale"], s["a"], s["b"], s["scale"], case["split_k"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    if own:
        return _library(s)
    return {"route": _route, "experts": _experts, "adapted": _adapted}[s["op"]](s)


def _library(s):
    if s["op"] == "route":
        from mxfp8_decode_gemm_amd import device as dv

        return dv.route(s["logits"], s["top_k"], score=s["score"], bias=s["bias"], groups=s["groups"],
                        top_groups=s["top_groups"], group_best=s["group_best"], renormalize=s["renormalize"],
                        scale=s["scale"])
    if s["op"] == "experts":
        return s["handle"](s["x"], s["ids"], s["weights"])
    return s["handle"](s["x"], s["ids"], x_scale=s["x_scale"])


def _route(s):
    """In 64 bits: neighbouring scores differ by less than 32 bits keep, and the order of equal ones is the index's."""
    v = s["logits"].double()
    score = torch.sigmoid(v) if s["score"] == "sigmoid" else torch.softmax(v, -1)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if s["groups"] > 1:
        t = v.shape[0]
        grouped = choice.view(t, s["groups"], -1)
        best = grouped.sort(dim=-1, descending=True).values[..., : s["group_best"]].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, : s["top_groups"]]
        keep = torch.zeros(t, s["groups"], dtype=torch.bool, device=v.device).scatter_(1, kept, True)
        choice = grouped.masked_fill(~keep.unsqueeze(-1), -torch.inf).view(t, -1)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, : s["top_k"]]
    weights = score.gather(1, ids)
    if s["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return ids.int(), (weights * s["scale"]).float()


def _decode(codes, scales):
    """The float32 values of MXFP8 codes and scale bytes (1..254: a scale byte is the exponent field of its value)."""
    v = codes.view(torch.float8_e4m3fn).float()
    step = (scales.int() << 23).view(torch.float32)
    return (v.view(*v.shape[:-1], -1, 32) * step.unsqueeze(-1)).view(v.shape)


def _experts(s):
    t, k = s["ids"].shape
    e = s["ids"].flatten().long()
    x = s["x"].float().repeat_interleave(k, 0).unsqueeze(-1)  # one row per (token, choice)
    gate, up = (_decode(s["w13"][e], s["w13_scale"][e]) @ x).chunk(2, 1)
    h = gate / (1 + torch.exp(-gate)) * up
    y = (_decode(s["w2"][e], s["w2_scale"][e]) @ h).view(t, k, -1)
    return (y * s["weights"].unsqueeze(-1)).sum(1).bfloat16()


def _adapted(s):
    m = s["x"].shape[0]
    x = s["x"].float() if s["x_scale"] is None else _decode(s["x"], s["x_scale"])
    xq = _decode(*_encode(x)) if s["x_scale"] is None else x
    base = xq @ _decode(s["w"], s["w_scale"]).t()
    some, a = s["ids"] >= 0, s["ids"].clamp_min(0).long()
    u = s["a"][a].float() @ x.unsqueeze(-1)
    delta = (s["b"][a].float() @ u).view(m, -1) * s["scale"][a].unsqueeze(-1)
    return (base + torch.where(some.unsqueeze(-1), delta, torch.zeros_like(delta))).bfloat16()


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _value64(codes, scales):
    """float64 values from the bits: sign, 4 exponent bits (bias 7), 3 mantissa bits; scale byte s is 2^(s - 127)."""
    c = codes.long()
    mant, ex = (c & 7).double(), (c >> 3) & 15
    mag = torch.where(ex == 0, mant * 2.0**-9, torch.ldexp(1 + mant / 8, ex - 7))
    v = torch.where(c >= 128, -mag, mag)
    ex = scales.long().repeat_interleave(32, -1) - 127
    return torch.ldexp(v, ex)


def _quantized64(x):
    """The values an MXFP8 encoding of the rows stands for, from float64 arithmetic alone."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp_min(2.0**-126) / 448)) - 1
    for _ in range(3):
        e = torch.where(448 * torch.exp2(e) < amax, e + 1, e)
    y = b / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0**-6))).clamp_min(-6) - 3)
    return (torch.round(y / step) * step * torch.exp2(e)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        v = s["logits"].double().cpu().numpy()
        if case["score"] == "sigmoid":
            score = 1 / (1 + np.exp(-v))
        else:
            score = np.exp(v - v.max(1, keepdims=True))
            score /= score.sum(1, keepdims=True)
        choice = score if s["bias"] is None else score + s["bias"].double().cpu().numpy()
        if case["groups"] > 1:
            t, g = v.shape[0], case["groups"]
            best = -np.sort(-choice.reshape(t, g, -1), -1)[..., : case["group_best"]].sum(-1)
            order = np.argsort(-best, 1, kind="stable")
            keep = np.zeros((t, g), bool)
            np.put_along_axis(keep, order[:, : case["top_groups"]], True, 1)
            choice = np.where(np.repeat(keep, v.shape[1] // g, 1), choice, -np.inf)
        ids = np.argsort(-choice, 1, kind="stable")[:, : case["top_k"]]
        weights = np.take_along_axis(score, ids, 1)
        if case["renormalize"]:
            weights = weights / weights.sum(1, keepdims=True)
        return ids.astype(np.int32), weights * case["scale"]
    if case["op"] == "experts":
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        x, ids, weights = s["x"].double(), s["ids"].cpu(), s["weights"].double()
        for e in sorted(set(ids.flatten().tolist())):
            t, j = (n.cuda() for n in (ids == e).nonzero(as_tuple=True))
            z = x[t] @ _value64(s["w13"][e], s["w13_scale"][e]).t()
            gate, up = z[:, : case["inter"]], z[:, case["inter"] :]
            y = (gate * torch.sigmoid(gate) * up) @ _value64(s["w2"][e], s["w2_scale"][e]).t()
            out.index_add_(0, t, y * weights[t, j].unsqueeze(-1))
        return out
    x = s["x"].double() if case["x"] == "bf16" else _value64(s["x"], s["x_scale"])
    shared = _quantized64(x) if case["x"] == "bf16" else x
    out = shared @ _value64(s["w"], s["w_scale"]).t()
    for row, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            out[row] += float(s["scale"][a]) * (s["b"][a].double() @ (s["a"][a].double() @ x[row]))
    return out
