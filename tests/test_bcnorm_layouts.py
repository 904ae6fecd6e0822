"""Layouts of the tensors that the norm and rotation of keys and queries takes: which
are read and written where they lie, which are copied, and which are refused."""
from __future__ import annotations

import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from layer_helpers import DT
from mamba_ssd_sequence_fwd_amd import _lib

# name: a tensor (tokens, heads, dim) made of randn, whose channels are not contiguous though its
# heads lie dim elements apart
ODD = {
    "broadcast channels": lambda r: r(6, 4, 64)[..., :1].expand(6, 4, 64),
    "broadcast channels and tokens": lambda r: r(4, 64)[..., :1].expand(6, 4, 64),
    "tokens in a row": lambda r: r(64, 4, 64).permute(2, 1, 0),
    "every 64th channel": lambda r: r(6, 64, 4, 64)[..., 0].transpose(1, 2),
    "one head, broadcast": lambda r: r(6, 1, 1).expand(6, 1, 64),
}
# name: such a tensor that can be read where it lies, and its row stride
PLAIN = {
    "contiguous": (lambda r: r(6, 4, 64), 256),
    "slice": (lambda r: r(6, 6, 64)[:, 1:5], 384),
    "batch of slices": (lambda r: r(2, 3, 6, 64)[:, :, 1:5], 384),
    "one head of several": (lambda r: r(6, 4, 64)[:, 2:3], 256),
    "every second token": (lambda r: r(12, 4, 64)[::2], 512),
    "no tokens": (lambda r: r(0, 4, 64), 256),
}


def as_kernel_reads(t, stride):
    """The rows at ``stride`` from t's first element, its heads and channels contiguous."""
    rows = t.shape[:-2].numel()
    return t.as_strided((rows, t.shape[-2] * t.shape[-1]), (stride, 1)).reshape(t.shape)


@pytest.mark.parametrize("name", ODD)
def test_strided_channels_are_copied_and_refused_as_outputs(name):
    t = ODD[name](torch.randn)
    assert _lib._head_rows(t) is None
    rows, stride = _lib._head_rows_in(t)
    assert rows is not t and torch.equal(as_kernel_reads(rows, stride), t)
    with pytest.raises(ValueError):
        _lib._head_rows_out(t, t, "B_out")


@pytest.mark.parametrize("name", PLAIN)
def test_rows_are_read_where_they_lie(name):
    make, stride = PLAIN[name]
    t = make(torch.randn)
    rows, got = _lib._head_rows_in(t)
    assert rows is t and got == stride and torch.equal(as_kernel_reads(rows, got), t)
    assert _lib._head_rows_out(t, t, "B_out") == (t, stride)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("name", ODD)
def test_strided_channels(name, dtype):
    """The same bits as of contiguous tensors, in every place an input can take; as an
    output refused."""
    g = torch.Generator("cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(DT[dtype])
    t = {k: ODD[name](r) for k in ("B", "C", "dB", "dC")}
    c = {k: v.contiguous() for k, v in t.items()}
    w = 1 + 0.1 * torch.randn(64, device="cuda", generator=g)
    kw = dict(positions=torch.arange(t["B"].shape[0], device="cuda"),
              freqs=0.5 ** torch.arange(16, device="cuda"), unit=True)
    print("[gpu] bc norm of %s %s" % (name, dtype), flush=True)
    got, want = ssd.bc_norm(t["B"], t["C"], w, w, **kw), ssd.bc_norm(c["B"], c["C"], w, w, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = ssd.bc_norm_backward(t["dB"], t["dC"], t["B"], t["C"], w, w, **kw)
    want = ssd.bc_norm_backward(c["dB"], c["dC"], c["B"], c["C"], w, w, **kw)
    assert all(torch.equal(got[k], want[k]) for k in want)
    for k in ("B_out", "C_out"):
        with pytest.raises(ValueError):
            ssd.bc_norm(c["B"], c["C"], w, w, **kw, **{k: t["B"]})
    for k in ("dB", "dC"):
        with pytest.raises(ValueError):
            ssd.bc_norm_backward(c["dB"], c["dC"], c["B"], c["C"], w, w, **kw, **{k: t["B"]})
