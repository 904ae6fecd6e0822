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
                                  [0] * 599 + [70]])
def test_fewer_tokens_than_sequences(dtype, lens):
    case = ([int(n) for n in lens], True, 4, 64, 64, 2, dtype, True)
    both_ways("%d tokens in %d sequences %s" % (sum(lens), len(lens), dtype), case, 2000)
