"""Sizes of the gated delta rule at the edges of what is allowed, on the host (nothing
is launched)."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SIZES = """if True:
    import ctypes
    import mamba_ssd_sequence_fwd_amd as ssd
    from mamba_ssd_sequence_fwd_amd import _lib
    lib, n = ssd.load(), ctypes.c_size_t(0)
    for dtype in (ssd.SSD_DTYPE_BF16, ssd.SSD_DTYPE_F32):
        for tokens, seqs in ((1, 2), (2, 3), (63, 64), (63, 1000), (1, 70000)):
            p = _lib.Problem(1, tokens, 4, 64, 64, 2, 0, seqs, dtype, 0)
            for size in (lib.ssd_delta_workspace_size, lib.ssd_delta_backward_workspace_size):
                assert size(p, ctypes.byref(n)) == ssd.SSD_OK and n.value > 0
    print("sized")
"""


def test_fewer_tokens_than_sequences():
    """The workspace of packed calls with fewer tokens than sequences (their mean length
    is below one). In a process of its own: a division by zero would end it."""
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "sized" in r.stdout, (r.returncode, r.stderr[-500:])
