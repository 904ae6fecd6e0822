"""The operators around the SSD layer where element offsets pass 32 bits: the
last rows against the same call on those rows alone (the same arithmetic per
element, so the same bits)."""
from __future__ import annotations

import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
TAIL = 150


def _room(gib):
    free = torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() - torch.cuda.memory_allocated()
    if free < gib << 30:
        pytest.skip("needs %d GiB of device memory" % gib)


def test_norm_rows_far_apart():
    _room(12)
    T, ch, stride = 2100, 512, 1 << 21                 # 2100 * 2^21 > 2^32 elements
    buf = torch.empty(T, stride, device="cuda", dtype=BF)
    x, z, dout, out, dx, dz = (buf[:, i * ch:(i + 1) * ch] for i in range(6))
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (x, z, dout):
        t.copy_(torch.randn(T, ch, device="cuda", generator=g))
    w = torch.randn(ch, device="cuda", generator=g)
    print("[gpu] norm with rows far apart", flush=True)
    _, kx, kz = ssd.group_norm_silu(x, w, None, z, groups=2, checkpoint=True, out=out)
    got = ssd.group_norm_silu_backward(dout, x, w, None, z, groups=2, dx=dx, dz=dz)
    near = [t.contiguous() for t in (x, z, dout)]
    want, nx, nz = ssd.group_norm_silu(near[0], w, None, near[1], groups=2, checkpoint=True)
    back = ssd.group_norm_silu_backward(near[2], near[0], w, None, near[1], groups=2)
    assert torch.equal(out, want) and torch.equal(kx.q, nx.q) and torch.equal(kz.q, nz.q)
    for k in ("dx", "dz", "dweight"):
        assert torch.equal(got[k], back[k]), k


def test_front_and_checkpoint_past_32_bits():
    _room(60)
    ch, x_dim, bc = 5376, 5120, 128
    T = (1 << 32) // ch + 200                          # T * ch > 2^32 elements
    g = torch.Generator(device="cuda").manual_seed(2)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)
    xbc = torch.zeros(T, ch, device="cuda", dtype=BF)
    xbc[-TAIL:] = rand(TAIL, ch).to(BF)
    w, b = rand(ch, 4), rand(ch)
    cu = torch.tensor([0, T - TAIL, T], dtype=torch.int32)
    one = torch.tensor([0, TAIL], dtype=torch.int32)
    print("[gpu] checkpoint and front past 32 bits", flush=True)
    x, B, C, _, kept = ssd.conv1d_silu(xbc, w, b, x_dim, bc, None, cu, want_history=False,
                                       checkpoint=True)
    saved = ssd.checkpoint_save(xbc)
    tail = ssd.checkpoint_save(xbc[-TAIL:].contiguous())
    for k in (kept, saved):
        assert torch.equal(k.q[-TAIL:], tail.q) and torch.equal(k.exponents[-TAIL:], tail.exponents)
    del saved
    assert torch.equal(kept.load()[-TAIL:], tail.load())
    want = ssd.conv1d_silu(xbc[-TAIL:].contiguous(), w, b, x_dim, bc, None, one)
    for name, u, v in zip("xBC", (x, B, C), want):
        assert torch.equal(u[-TAIL:], v), name
    again = ssd.conv1d_silu(kept, w, b, x_dim, bc, None, cu, x=x, B=B, C=C)
    want = ssd.conv1d_silu(tail, w, b, x_dim, bc, None, one)
    for name, u, v in zip("xBC", again, want):
        assert torch.equal(u[-TAIL:], v), name
    # the backward pass; x, B and C serve as its gradients
    for src, end in ((xbc, xbc[-TAIL:].contiguous()), (kept, tail)):
        got = ssd.conv1d_silu_backward(src, w, b, x, B, C, None, cu)
        alone = ssd.conv1d_silu_backward(end, w, b, *(t[-TAIL:].contiguous() for t in (x, B, C)),
                                         None, one)
        assert torch.equal(got["dxbc"][-TAIL:], alone["dxbc"])
        del got
