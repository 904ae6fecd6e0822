"""Inputs and bounds shared by the GPU tests of the operators around the SSD
layer.

Bounds, per element: with u = 2^-24 (half a step of fp32), an fp32 result is
within C u S of the oracle's, S being the sum of the magnitudes of the terms
it is made of (the oracle gives it) and C counting the roundings each term
goes through. A bf16 output is that value rounded once more, by at most 2^-8
of it (half a step, eps / 2).

C = 160 for the norm: silu's exponent argument (|z| < 7 here) and its two
hardware functions 15, the product 1, squares and the sum of up to 16 + 14
levels 63, halved by the root, the division and products 5; twice the 16 + 30
of a mean that is taken off; the second silu 15.
C = 512 for its gradients: h and g at 160 each, their product's mean through
the same sums, and up to 32 rows summed in turn.
C = 160 for the front's gradients: pre through K + 1 products and sums, silu'
through the same functions, K + 1 terms, up to 64 tokens summed in turn.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rows(rng, n, ch, dtype, lead=0, pad=0, spread=0.5):
    """(device tensor (n, ch) in rows of lead + ch + pad, its fp64 values)."""
    v = rng.standard_normal((n, lead + ch + pad)) * np.exp(
        spread * rng.standard_normal((1, lead + ch + pad)))
    t = torch.from_numpy(v.astype(np.float32)).to(DT[dtype])
    return t.cuda()[:, lead:lead + ch], t[:, lead:lead + ch].double().numpy()


def check(name, got, want, size, dtype, C):
    """Every element within its bound (``dtype`` of the output)."""
    g = got.detach().double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(g).all(), name
    err = np.abs(g - want)
    bound = C * U * size + (2.0 ** -8 if dtype == "bf16" else U) * np.abs(want) + 1e-38
    worst = float((err / bound).max()) if err.size else 0.0
    print("  %-10s max |err| %.2e, %.2f of its bound" % (name, err.max() if err.size else 0.0, worst),
          flush=True)
    assert worst <= 1.0, (name, worst)
