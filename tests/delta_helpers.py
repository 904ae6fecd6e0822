"""Inputs and bounds of the tests of the gated delta rule.

Bounds, in the Frobenius norm of a tensor (||got - ref|| <= bound * ||ref||), u =
eps / 2 of the type. Keys of unit length and 0 <= beta <= 2 make every token's
transition a contraction, so an error that enters the state does not grow.

fp32: a value goes through at most five products in a row (K S, T R, M U, K^T U
and the state's next K S), each a sum of up to 256 terms taken in turn, whose
rounding errors of u add to 16 u (independent signs): 5 * 16 = 80 u.
bf16, states and dinitial_state: what enters them is held in two bf16, off by at
most 2^-17 (the residual of a half step of 2^-8, rounded again: less than
2^-8 * 2^-9), in three operands in a row (S, R, U): 3 * 2^-17, more than the
fp32 sums add.
bf16, y and the gradients: rounded once themselves, by at most u = 2^-8, after sums of
products of which at most two operands are rounded to bf16 (S, M and U; for the
gradients U, dR, S, dS and the pair matrices). Those errors are uniform up to u,
u / sqrt(3) in the root mean square, and of independent signs: sqrt(2) u / sqrt(3) of
the terms' norm, which is taken to be at most twice the sum's (unit keys and random
values cancel no further): u (1 + 2 sqrt(2 / 3)) = 2.6 u.
A single element is held to 8 times that of the largest of the tensor.
"""
from __future__ import annotations

import numpy as np
import torch

import mamba_ssd_sequence_fwd_amd as ssd

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
BOUND = {"bf16": 2.6 * 2.0 ** -8, "fp32": 80 * 2.0 ** -24}
STATE = {"bf16": 3 * 2.0 ** -17, "fp32": 80 * 2.0 ** -24}

CASES = {
    # name: (sequence lengths, packed, H, P, N, G, dtype, initial state)
    "one-token": ([1, 1, 1], False, 4, 64, 128, 1, "bf16", True),
    "one-chunk-less-one": ([63, 63], False, 2, 64, 64, 2, "bf16", False),
    "one-chunk": ([64], False, 3, 32, 16, 1, "bf16", True),
    "one-chunk-and-one": ([65, 65], False, 6, 128, 128, 2, "bf16", True),
    "P16-N48": ([100, 100, 100], False, 5, 16, 48, 1, "bf16", True),
    "P32-N80-G3": ([130, 130], False, 9, 32, 80, 3, "bf16", False),
    "N176": ([190], False, 4, 64, 176, 2, "bf16", True),
    "P128-N256": ([150, 150], False, 2, 128, 256, 1, "bf16", True),
    "P16-N256-G2": ([77], False, 2, 16, 256, 2, "bf16", False),
    "packed": ([70, 0, 1, 64, 0, 200, 63, 129], True, 6, 64, 128, 1, "bf16", True),
    "packed-empty-ends": ([0, 0, 128, 5, 0], True, 4, 128, 64, 4, "bf16", True),
    "packed-P16": ([3, 9, 1, 0, 30, 65], True, 2, 16, 32, 1, "bf16", False),
    "many-heads-a-group": ([90, 90], False, 40, 64, 64, 1, "bf16", False),
    "segments": ([1100], False, 2, 64, 64, 1, "bf16", True),
    "segments-N128": ([1283, 1283], False, 4, 128, 128, 2, "bf16", True),
    "segments-N256": ([1200], False, 2, 128, 256, 1, "bf16", True),
    "segments-P16-N176": ([1250], False, 3, 16, 176, 3, "bf16", False),
    "segments-packed": ([2500, 0, 1999, 1], True, 2, 32, 48, 1, "bf16", True),
    "long-N128": ([3000], False, 2, 128, 128, 1, "bf16", True),
    "long-N256": ([3200], False, 1, 128, 256, 1, "bf16", True),
    "long-P16-N176": ([3000], False, 2, 16, 176, 2, "bf16", False),
    "ordered-33": ([(37 * i) % 101 for i in range(33)], True, 3, 128, 32, 1, "bf16", True),
    "ordered-64": ([(61 * i) % 130 if i % 5 else 0 for i in range(64)], True, 2, 32, 64, 2, "bf16",
                   False),
    "ordered-512": ([(i * i) % 9 for i in range(512)], True, 2, 16, 16, 1, "bf16", True),
    "not-ordered-513": ([(i * i) % 7 for i in range(513)], True, 2, 16, 16, 1, "bf16", True),
    "one-token-fp32": ([1, 1], False, 4, 64, 128, 1, "fp32", True),
    "one-chunk-and-one-fp32": ([65], False, 6, 32, 64, 2, "fp32", False),
    "P16-N48-fp32": ([100, 100], False, 5, 16, 48, 1, "fp32", True),
    "N176-fp32": ([190], False, 2, 64, 176, 1, "fp32", True),
    "P128-N256-fp32": ([150], False, 2, 128, 256, 1, "fp32", True),
    "packed-fp32": ([70, 0, 1, 64, 0, 200], True, 4, 128, 128, 2, "fp32", True),
    "long-fp32": ([700], False, 3, 64, 64, 3, "fp32", False),
}


def inputs(case, seed, rate=1.0, top=1.0):
    """CPU tensors in the call's dtype: unit keys and queries, g = -rate * softplus,
    beta in (0, top)."""
    lens, packed, H, P, N, G, dtype, state = case
    T, S, dt = sum(lens), len(lens), DT[dtype]
    rng = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=rng)
    unit = lambda v: v / v.norm(dim=-1, keepdim=True).clamp_min(1e-6)
    d = dict(x=r(T, H, P), g=-rate * torch.nn.functional.softplus(r(T, H) - 2),
             beta=top * torch.sigmoid(r(T, H)), B=unit(r(T, G, N)), C=unit(r(T, G, N)),
             dy=r(T, H, P))
    d = {k: v.to(dt) for k, v in d.items()}
    d["h0"] = 0.5 * r(S, H, P, N) if state else None
    d["dhT"] = 0.2 * r(S, H, P, N) if state else None
    return d


def on_gpu(d, case):
    """Device tensors with the call's leading axes, and cu_seqlens (host) or None."""
    lens, packed = case[0], case[1]
    lead = (1, sum(lens)) if packed else (len(lens), lens[0])
    t = {k: v.cuda() if k in ("h0", "dhT") else v.reshape(lead + v.shape[1:]).cuda()
         for k, v in d.items() if v is not None}
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32) if packed else None
    return t, cu


def forward(t, cu, **kw):
    return ssd.delta_forward(t["x"], t["g"], t["beta"], t["B"], t["C"], t.get("h0"), cu, **kw)


def backward(t, cu, **kw):
    return ssd.delta_backward(t["x"], t["g"], t["beta"], t["B"], t["C"], t.get("h0"), t["dy"],
                              t.get("dhT"), cu, **kw)


def check(name, got, want, bound):
    g = got.detach().double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(g).all(), name
    if g.size == 0:
        return
    norm, top = np.linalg.norm(want), np.abs(want).max()
    err, worst = np.linalg.norm(g - want), np.abs(g - want).max()
    print("  %-15s %.2f of its bound, one element %.2f" %
          (name, err / (bound * norm + 1e-30), worst / (8 * bound * top + 1e-30)), flush=True)
    assert err <= bound * norm, (name, err / norm)
    assert worst <= 8 * bound * top, (name, worst / top)
