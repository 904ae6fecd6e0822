"""The gated delta rule on the GPU at the edges of what is allowed, against the fp64
oracle; inputs and bounds in delta_helpers."""
from __future__ import annotations

import pytest
import torch

from delta_helpers import BOUND, STATE, backward, check, forward, inputs, on_gpu
from oracle.delta import delta_backward, delta_rule

pytestmark = pytest.mark.gpu
GRADS = ("dx", "dg", "dbeta", "dB", "dC")


def both_ways(name, case, seed):
    """Forward and backward of a case against the oracle."""
    d = inputs(case, seed)
    t, cu = on_gpu(d, case)
    print("[gpu] delta %s" % name, flush=True)
    y, h = forward(t, cu)
    g = backward(t, cu)
    torch.cuda.synchronize()
    dtype = case[6]
    want, hw = delta_rule(d["x"], d["g"], d["beta"], d["B"], d["C"], d["h0"], case[0])
    check("y", y, want, BOUND[dtype])
    check("final_state", h, hw, STATE[dtype])
    want = delta_backward(d["x"], d["g"], d["beta"], d["B"], d["C"], d["h0"], case[0], d["dy"],
                          d["dhT"])
    for k in GRADS:
        check(k, g[k], want[k], BOUND[dtype])
    check("dinitial_state", g["dinitial_state"], want["dinitial_state"], STATE[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[0, 1, 0], [1, 0, 0, 1, 0], [i % 3 == 1 for i in range(100)],
                                  [0] * 99 + [70]])
def test_fewer_tokens_than_sequences(dtype, lens):
    case = ([int(n) for n in lens], True, 4, 64, 64, 2, dtype, True)
    both_ways("%d tokens in %d sequences %s" % (sum(lens), len(lens), dtype), case, 2000)


def _many(n):
    """n short sequences: chunks enough for the rules that share a group's heads out, and a few
    that are whole or one past."""
    return [130 if i == 7 else 64 if i % 50 == 0 else 65 if i % 50 == 25 else i * i % 3
            for i in range(n)]


# name: (case, heads a wave takes in turn for the triangular matrices forwards and backwards,
#        and parts of a group's heads in the gradients)
MANY = {
    "13 heads a group": ((_many(256), True, 13, 64, 128, 1, "bf16", True), (2, 2), [5, 5, 3]),
    "11 heads a group, not ordered": ((_many(600), True, 11, 64, 64, 1, "bf16", False), (3, 3),
                                      [11]),
    "P 128, 10 heads": ((_many(256), True, 10, 128, 112, 1, "bf16", True), (1, 2), [4, 4, 2]),
    "P 128, 2 heads a group": ((_many(256), True, 8, 128, 80, 4, "bf16", True), (2, 1), [2]),
    "3 heads a group": ((_many(256), True, 12, 32, 64, 4, "bf16", True), (3, 1), [3]),
    "N 176, 13 heads": ((_many(256), True, 13, 64, 176, 1, "bf16", False), (2, 2), [5, 5, 3]),
    "P 128, N 144, 9 heads": ((_many(256), True, 9, 128, 144, 1, "bf16", True), (1, 2), [3, 3, 3]),
    "P 32, 2 groups of 5": ((_many(256), True, 10, 32, 48, 2, "bf16", True), (2, 2), [5]),
    "fp32, 9 heads": ((_many(256), True, 9, 32, 64, 1, "fp32", True), (2, 2), None),
    "fp32, P 128, 2 groups of 5": ((_many(256), True, 10, 128, 128, 2, "fp32", False), (2, 2),
                                   None),
    "fp32, a head a group": ((_many(64), True, 3, 64, 64, 3, "fp32", True), (1, 1), None),
}


def _shares(case):
    """The launches' rules for sharing out a group's heads: how many a wave takes in turn for the
    triangular matrices, and the parts that the gradients (bf16) take."""
    lens, packed, H, P, N, G, dtype, _ = case
    slots = sum(lens) // 64 + len(lens)
    heads, groups = H // G, slots * G
    few = dtype == "bf16"                       # forwards
    waves = 1 if few and heads <= 3 else min(heads, 2) if heads < 3 else 4
    ahead = -(-heads // (waves * max((1024 if few else 768) // groups, 1)))
    waves = min(heads, 2) if heads < 3 else 4
    back = -(-heads // (waves * max(768 // groups, 1)))
    own = -(-heads // max(1, min(heads, 1024 // groups)))
    return (ahead, back), [min(own, heads - k) for k in range(0, heads, own)]


@pytest.mark.parametrize("name", MANY)
def test_heads_in_turn(name):
    """Several heads taken in turn by a wave or workgroup, with a last part that is shorter."""
    case, per, parts = MANY[name]
    assert _shares(case)[0] == per and (parts is None or _shares(case)[1] == parts)
    both_ways(name, case, 2100 + sorted(MANY).index(name))
