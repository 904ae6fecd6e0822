"""How many bits the gated delta rule's bf16 calls keep: y and the gradients are what 32-bit
arithmetic gives, rounded once, and the fp32 states are 32-bit arithmetic's.

What a bf16 output is off by beyond half a step of its type is what was off before it was
rounded (excess). Bounds, in the Frobenius norm, with u = 2^-24 and inputs as in
delta_helpers (a contraction, so that an error which enters a state does not grow):

y: its terms are products of S, M and U, which are held in two bf16 there (each off by at
most 2^-17: a residual below 2^-8, whose own half step is 2^-17), without the product of two
residuals (2^-8 each: 2^-16 of a term). 3 * 2^-17 + 2^-16 = 5 * 2^-17 of the terms' norm,
which is at most twice the sum's (unit keys and random values cancel no further):
10 * 2^-17.
Gradients: a pair matrix is a product of two such operands (2 * 2^-17 + 2^-16), itself held in
two bf16 (2^-17); the states' products are of two of them: at most 5 * 2^-17 of the terms as
well.
States and dinitial_state: what enters them is held in three bf16 (2^-26, nothing beside u).
A product adds up to 24 results of a matrix instruction in turn, each rounded by up to u of
independent sign: sqrt(24 / 3) u = 2.8 u; five products in a row sqrt(5) of that, 6.3 u; the
decays' hardware exponential and the rounding of its argument (up to 16 in base 2) 4 u each:
together sqrt(6.3^2 + 4^2 + 4^2) u = 8.5 u, held to 16 u.
A single element is held to 8 times that of the largest of the tensor, as in delta_helpers.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from delta_helpers import CASES, backward, forward, inputs, on_gpu
from oracle.delta import delta_backward, delta_rule

pytestmark = pytest.mark.gpu
EXCESS, STATE = 10 * 2.0 ** -17, 16 * 2.0 ** -24
NAMES = ["one-token", "one-chunk-and-one", "P16-N48", "P32-N80-G3", "N176", "P128-N256", "packed",
         "many-heads-a-group", "segments-N128", "segments-N256", "segments-P16-N176",
         "segments-packed", "ordered-64"]


def half_step(want):
    """Half the distance of neighbouring bf16 values at ``want``."""
    return np.ldexp(1.0, np.frexp(want)[1] - 9)


def close(name, got, want, bound, rounded):
    g = got.detach().double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(g).all(), name
    if g.size == 0:
        return
    off = np.abs(g - want)
    if rounded:
        off = np.maximum(off - half_step(want), 0)
    norm, top = np.linalg.norm(want), np.abs(want).max()
    err, worst = np.linalg.norm(off), off.max()
    print("  %-15s %.2f of its bound, one element %.2f" %
          (name, err / (bound * norm + 1e-30), worst / (8 * bound * top + 1e-30)), flush=True)
    assert err <= bound * norm, (name, err / norm)
    assert worst <= 8 * bound * top, (name, worst / top)


@pytest.mark.parametrize("name", NAMES)
def test_forward(name):
    case = CASES[name]
    d = inputs(case, 2200 + NAMES.index(name))
    t, cu = on_gpu(d, case)
    print("[gpu] delta bits forward %s" % name, flush=True)
    y, h = forward(t, cu)
    torch.cuda.synchronize()
    want, hw = delta_rule(d["x"], d["g"], d["beta"], d["B"], d["C"], d["h0"], case[0])
    close("y", y, want, EXCESS, True)
    close("final_state", h, hw, STATE, False)


@pytest.mark.parametrize("name", NAMES)
def test_backward(name):
    case = CASES[name]
    d = inputs(case, 2300 + NAMES.index(name))
    t, cu = on_gpu(d, case)
    print("[gpu] delta bits backward %s" % name, flush=True)
    g = backward(t, cu)
    torch.cuda.synchronize()
    want = delta_backward(d["x"], d["g"], d["beta"], d["B"], d["C"], d["h0"], case[0], d["dy"],
                          d["dhT"])
    for k in ("dx", "dg", "dbeta", "dB", "dC"):
        close(k, g[k], want[k], EXCESS, True)
    close("dinitial_state", g["dinitial_state"], want["dinitial_state"], STATE, False)


@pytest.mark.parametrize("name", ["packed", "segments"])
def test_resets(name):
    """Decays behind a reset, where the sums of log decays are large and their differences
    small: two floats hold them."""
    case = CASES[name]
    d = inputs(case, 2400, rate=0.2)
    d["g"][::37, 0] = -1000.0
    d["g"][5, 1] = -1000.0
    t, cu = on_gpu(d, case)
    print("[gpu] delta bits resets %s" % name, flush=True)
    y, h = forward(t, cu)
    g = backward(t, cu)
    torch.cuda.synchronize()
    args = [d[k] for k in ("x", "g", "beta", "B", "C", "h0")]
    want, hw = delta_rule(*args, case[0])
    close("y", y, want, EXCESS, True)
    close("final_state", h, hw, STATE, False)
    want = delta_backward(*args, case[0], d["dy"], d["dhT"])
    for k in ("dx", "dg", "dbeta", "dB", "dC"):
        close(k, g[k], want[k], EXCESS, True)
    close("dinitial_state", g["dinitial_state"], want["dinitial_state"], STATE, False)
