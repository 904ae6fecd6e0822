"""Sizes and refusals of the gated delta rule at the edges of what is allowed, on the
host (nothing is launched)."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from mamba_ssd_sequence_fwd_amd import _lib

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


def _m(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _kept(t):
    """A Checkpoint with the shape, dtype and device of t."""
    q = torch.empty(t.shape, dtype=torch.int8, device=t.device)
    exponents = torch.empty(t.shape[:-1] + (-(-t.shape[-1] // 32),), dtype=torch.uint8,
                            device=t.device)
    return ssd.Checkpoint(q, exponents, t.dtype)


@pytest.mark.parametrize("call,names", [
    ("forward", ("x", "g", "beta", "B", "C", "initial_state", "cu_seqlens", "y", "final_state")),
    ("backward", ("x", "g", "beta", "B", "C", "initial_state", "cu_seqlens", "dy", "dfinal_state")),
    ("step", ("x", "g", "beta", "B", "C", "state", "y"))])
def test_a_checkpoint_is_refused_by_name(call, names, monkeypatch):
    """A Checkpoint has a tensor's shape, dtype and device: it is named where one stands in a
    tensor's place, whatever that place is."""
    monkeypatch.setattr(_lib, "_on_gpu", lambda dev: None)
    lead = (2,) if call == "step" else (2, 9)
    like = dict(x=_m(*lead, 8, 64), g=_m(*lead, 8), beta=_m(*lead, 8), B=_m(*lead, 2, 32),
                C=_m(*lead, 2, 32))
    state = _m(2, 8, 64, 32, dtype=torch.float32)
    like.update(y=like["x"], dy=like["x"], cu_seqlens=_m(1, 8, dtype=torch.float32), state=state,
                initial_state=state, final_state=state, dfinal_state=state)
    needed = ("x", "g", "beta", "B", "C") + {"forward": (), "backward": ("initial_state", "dy"),
                                             "step": ("state",)}[call]
    for name in names:
        t = {k: like[k] for k in needed}
        t[name] = _kept(like[name])
        with pytest.raises(ValueError, match="^%s is a Checkpoint" % name):
            getattr(ssd, "delta_" + call)(**t)


def test_workspace_without_groups_of_heads():
    """Backward in fp32: per chunk and head three matrices of 64 x 64, the states at its ends,
    U and dR. Gradients of keys and queries by the head are kept where a group has several to
    add up, and nowhere else."""
    lib, n = ssd.load(), ctypes.c_size_t(0)
    tokens, H, P, N = 640, 6, 64, 128
    own = 4 * (tokens // 64) * H * (3 * 64 * 64 + 2 * P * N + 2 * 64 * P)
    for G, by_head in ((6, 0), (3, 1), (1, 1)):
        p = _lib.Problem(1, tokens, H, P, N, G, 0, 0, ssd.SSD_DTYPE_F32, 0)
        assert lib.ssd_delta_backward_workspace_size(p, ctypes.byref(n)) == ssd.SSD_OK
        assert n.value == own + by_head * 2 * 4 * tokens * H * N
