"""Inputs of the tests of the products of any number of rows: seeded codes, and device copies."""

import numpy as np
import torch

from oracle import rows as oracle


def weights(rng, form, *shape):
    """Random codes and scale bytes of [..., n, k]: every E2M1 code; e4m3 codes of normals quantized per 32."""
    *lead, n, k = shape
    if form == "mxfp4":
        return (rng.integers(0, 256, (*lead, n, k // 2), dtype=np.uint8),
                rng.integers(118, 126, (*lead, n, k // 32), dtype=np.uint8))
    from workloads import generate

    v = rng.standard_normal((int(np.prod([*lead, n])), k)) * k**-0.5
    q, s = generate.quantize_mxfp8(v)
    return q.reshape(*lead, n, k), s.reshape(*lead, n, k // 32)


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def close(got, exact, slack):
    """Whether every BF16 value is within the bound of the exact one."""
    return (np.abs(f64(got) - exact) <= oracle.bf16_bound(exact, slack)).all()
