"""8-bit checkpoints on the GPU: whole tensors, and written and read by the
convolution front, bit for bit against the fp64 oracle of the form."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
import ssd_inputs as si
from layer_helpers import rows
from oracle.checkpoint import kept, quantise
from oracle.conv import conv_front, dense_bounds, varlen_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,ch,dtype,lead,pad", [
    (1, 8, "bf16", 0, 0), (5, 40, "fp32", 0, 0), (257, 96, "bf16", 8, 24), (33, 5376, "bf16", 0, 0),
    (64, 1000, "fp32", 4, 4), (3, 72, "bf16", 0, 8),
])
def test_save_and_load(n, ch, dtype, lead, pad):
    rng = np.random.default_rng(n + ch)
    t, v = rows(rng, n, ch, dtype, lead, pad, spread=3.0)
    print("[gpu] checkpoint %d x %d %s" % (n, ch, dtype), flush=True)
    k = ssd.checkpoint_save(t)
    back = k.load()
    wide = torch.full((n, ch + 16), 9.0, dtype=t.dtype, device="cuda")
    assert k.load(out=wide[:, 8:8 + ch]).data_ptr() == wide[:, 8:].data_ptr()
    torch.cuda.synchronize()
    q, byte = quantise(v)
    assert np.array_equal(k.q.cpu().numpy(), q) and np.array_equal(k.exponents.cpu().numpy(), byte)
    assert np.array_equal(back.double().cpu().numpy(), kept(v))
    assert torch.equal(wide[:, 8:8 + ch], back)
    assert (wide[:, :8] == 9).all() and (wide[:, 8 + ch:] == 9).all()


def test_special_blocks():
    """Zeros, ties, the ends of both types, infinities and NaN."""
    v = np.zeros((12, 64), np.float32)
    v[1, :3] = 127.0, 0.5, 1.5
    v[2, :2] = 127.5, 1.0
    v[3, 40] = np.finfo(np.float32).max
    v[4, :] = np.float32(1e-45)
    v[5, :2] = np.float32(2.0 ** -119), np.float32(-2.0 ** -126)
    v[6, 5], v[6, 33] = np.inf, 2.0
    v[7, 9] = np.nan
    v[8, 1], v[8, 0] = -np.inf, 1.0
    v[9, :] = -np.linspace(1, 127, 64)
    v[10, :2] = 1.9921875, -1.9921874
    v[11, :2] = 1e30, 1e-30
    print("[gpu] checkpoint special blocks", flush=True)
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(v).to(dtype)
        k = ssd.checkpoint_save(t.cuda())
        back = k.load()
        torch.cuda.synchronize()
        q, byte = quantise(t.double())
        assert np.array_equal(k.q.cpu().numpy(), q), dtype
        assert np.array_equal(k.exponents.cpu().numpy(), byte), dtype
        assert np.array_equal(back.double().cpu().numpy(), kept(t.double()), equal_nan=True)


def test_empty_filled_and_twice():
    print("[gpu] checkpoint reuse", flush=True)
    e = ssd.checkpoint_save(torch.empty(0, 64, device="cuda"))
    assert e.load().shape == (0, 64)
    t = torch.randn(2, 7, 64, device="cuda").to(torch.bfloat16)
    k = ssd.checkpoint_save(t)
    u = torch.randn(2, 7, 64, device="cuda").to(torch.bfloat16)
    assert ssd.checkpoint_save(u, checkpoint=k) is k
    again = ssd.checkpoint_save(k.load())       # what 8 bits hold, they hold again
    torch.cuda.synchronize()
    assert torch.equal(again.load(), k.load()) and k.shape == (2, 7, 64)
    with pytest.raises(ValueError, match="fill"):
        ssd.checkpoint_save(torch.randn(3, 64, device="cuda"), checkpoint=k)
    with pytest.raises(ValueError, match="multiple of 8"):
        ssd.checkpoint_save(torch.randn(3, 60, device="cuda"))


def test_offsets_past_32_bits():
    """Rows whose offsets pass 2^32 elements, on both sides."""
    n, ch = (1 << 17) + 3, 1 << 15
    print("[gpu] checkpoint past 32-bit offsets", flush=True)
    t = torch.zeros(n, ch, dtype=torch.bfloat16, device="cuda")
    t[-3:] = torch.randn(3, ch, device="cuda")
    k = ssd.checkpoint_save(t)
    small = ssd.checkpoint_save(t[-3:].clone())
    torch.cuda.synchronize()
    assert torch.equal(k.q[-3:], small.q) and torch.equal(k.exponents[-3:], small.exponents)
    assert torch.equal(k.load(out=t)[-3:], small.load())


FRONT = {
    # name: (batch, seqlen, seq_lens, x_dim, bc_dim, K, dtype, lead, pad); channel counts that
    # are and are not whole blocks, interior and general tiles
    "bf16-K4-dense": (2, 300, None, 128, 32, 4, "bf16", 0, 0),
    "fp32-K3-odd-groups": (3, 65, None, 72, 16, 3, "fp32", 0, 0),
    "bf16-K2-packed-slice": (1, 0, [33, 0, 31, 64, 1, 2], 40, 8, 2, "bf16", 16, 8),
    "fp32-K4-eight-channels": (2, 40, None, 8, 0, 4, "fp32", 0, 0),
    "bf16-K4-many-groups": (1, 90, None, 2600, 40, 4, "bf16", 0, 0),
}


@pytest.mark.parametrize("hist", [False, True])
@pytest.mark.parametrize("name", sorted(FRONT))
def test_conv_front_saves_and_recomputes(name, hist):
    """checkpoint=True changes no output and keeps the oracle's 8 bits; the
    front from them equals the front of their values."""
    batch, seqlen, lens, x_dim, bc_dim, K, dtype, lead, pad = FRONT[name]
    inp = si.make_conv_inputs(batch, seqlen, x_dim, bc_dim, K, dtype, seed=4800, seq_lens=lens,
                              history=hist, lead_cols=lead, pad_cols=pad)
    ch = x_dim + 2 * bc_dim
    xbc = inp["xbc_full"].cuda()[:, lead:lead + ch]
    if lens is None:
        xbc = xbc.view(batch, seqlen, ch)
    args = (inp["weight"].cuda(), inp["bias"].cuda(), x_dim, bc_dim,
            inp["history"].cuda() if hist else None, inp["cu_seqlens"])
    print("[gpu] conv front checkpoint %s" % name, flush=True)
    plain = ssd.conv1d_silu(xbc, *args)
    saved = ssd.conv1d_silu(xbc, *args, checkpoint=True)
    again = ssd.conv1d_silu(saved[4], *args)
    direct = ssd.conv1d_silu(saved[4].load(), *args)
    torch.cuda.synchronize()
    bounds = dense_bounds(batch, seqlen) if lens is None else \
        varlen_bounds(inp["cu_seqlens"].tolist())
    q, byte = quantise(inp["xbc"])
    assert np.array_equal(saved[4].q.reshape(-1, ch).cpu().numpy(), q)
    assert np.array_equal(saved[4].exponents.reshape(inp["T"], -1).cpu().numpy(), byte)
    assert torch.equal(saved[3], plain[3]) and again[3] is None
    want = conv_front(kept(inp["xbc"]), inp["weight"], inp["bias"], bounds, x_dim, bc_dim,
                      inp["history"])
    # one instantiation may fuse a product and sum where another does not: an
    # output may then round to its neighbour (a step, 2^-7 in bf16, of it)
    step, atol = (2.0 ** -7, 2e-5) if dtype == "bf16" else (1e-5, 1e-5)
    for k in range(3):
        assert torch.allclose(saved[k].float(), plain[k].float(), rtol=step, atol=atol), k
        assert torch.allclose(again[k].float(), direct[k].float(), rtol=step, atol=atol), k
        g = again[k].double().cpu().numpy().reshape(want[k].shape)
        rtol = 2.0 ** -8 if dtype == "bf16" else 1e-5
        assert (np.abs(g - want[k]) <= atol + rtol * np.abs(want[k])).all(), k


@pytest.mark.parametrize("hist", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_conv_front_without_tokens_is_kept(packed, hist):
    """No tokens and checkpoint=True: the history passes through (zeros without
    one), the checkpoint is empty, and x, B and C come back from it empty."""
    nseq, x_dim, bc_dim, K = 4, 64, 16, 4
    ch = x_dim + 2 * bc_dim
    lead = (0,) if packed else (nseq, 0)
    g = torch.Generator().manual_seed(4900)
    w, b = torch.randn(ch, K, generator=g).cuda(), torch.randn(ch, generator=g).cuda()
    h = torch.randn(nseq, K - 1, ch, generator=g).to(torch.bfloat16).cuda() if hist else None
    cu = torch.zeros(nseq + 1, dtype=torch.int32, device="cuda") if packed else None
    xbc = torch.empty(lead + (ch,), dtype=torch.bfloat16, device="cuda")
    print("[gpu] conv front without tokens, kept", flush=True)
    x, B, C, out, kept_ = ssd.conv1d_silu(xbc, w, b, x_dim, bc_dim, h, cu, checkpoint=True)
    given = ssd.conv1d_silu(xbc, w, b, x_dim, bc_dim, h, cu, checkpoint=kept_)
    again = ssd.conv1d_silu(kept_, w, b, x_dim, bc_dim, h, cu)
    torch.cuda.synchronize()
    want = h if hist else torch.zeros(nseq, K - 1, ch, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(out, want) and torch.equal(given[3], want) and again[3] is None
    assert kept_.shape == lead + (ch,) and kept_.exponents.shape == lead + (3,)
    assert given[4] is kept_ and kept_.load().shape == lead + (ch,)
    for got in ((x, B, C), again[:3]):
        assert [t.shape for t in got] == [lead + (n,) for n in (x_dim, bc_dim, bc_dim)]


def test_conv_from_a_checkpoint_does_not_look_at_the_input_stride():
    """The C calls with in_stride 0 and xbc NULL: what the binding's calls give."""
    x_dim, bc_dim, K, L = 64, 16, 4, 37
    ch = x_dim + 2 * bc_dim
    g = torch.Generator().manual_seed(4901)
    w, b = torch.randn(ch, K, generator=g).cuda(), torch.randn(ch, generator=g).cuda()
    kept_ = ssd.checkpoint_save(torch.randn(2, L, ch, generator=g).to(torch.bfloat16).cuda())
    d = [torch.randn(2, L, n, generator=g).to(torch.bfloat16).cuda()
         for n in (x_dim, bc_dim, bc_dim)]
    print("[gpu] conv front from a checkpoint, in_stride 0", flush=True)
    want = ssd.conv1d_silu(kept_, w, b, x_dim, bc_dim)[:3]
    wg = ssd.conv1d_silu_backward(kept_, w, b, *d)
    p = ssd.ConvProblem(2, L, 0, x_dim, bc_dim, K, 0, ssd.SSD_DTYPE_BF16, 0)
    out = [torch.zeros_like(t) for t in want]
    lib, stream = ssd.load(), torch.cuda.current_stream().cuda_stream
    assert lib.ssd_conv1d_silu_checkpoint(p, None, kept_.arg(), w.data_ptr(), b.data_ptr(), None,
                                          None, *(t.data_ptr() for t in out), None,
                                          stream) == ssd.SSD_OK
    n = ctypes.c_size_t(0)
    assert lib.ssd_conv1d_silu_backward_workspace_size(p, ctypes.byref(n)) == ssd.SSD_OK
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    dxbc, dw, db = torch.zeros_like(wg["dxbc"]), torch.zeros_like(w), torch.zeros_like(b)
    assert lib.ssd_conv1d_silu_backward(p, None, kept_.arg(), w.data_ptr(), b.data_ptr(), None,
                                        None, *(t.data_ptr() for t in d), None, dxbc.data_ptr(),
                                        ch, dw.data_ptr(), db.data_ptr(), None, ws.data_ptr(),
                                        n.value, stream) == ssd.SSD_OK
    torch.cuda.synchronize()
    for got, ref in zip(out + [dxbc, dw, db], list(want) + [wg[k] for k in ("dxbc", "dweight",
                                                                             "dbias")]):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_conv_front_outputs_do_not_depend_on_the_checkpoint(dtype, K, bias):
    """Two kernels, the same sums in the same order: keeping the input changes no
    bit of x, B, C and the history, and x, B and C from the checkpoint are those
    of its values."""
    print("[gpu] conv front with and without a checkpoint %s K=%d" % (dtype, K), flush=True)
    for batch, seqlen, lens, x_dim, bc_dim, hist in (
            (3, 515, None, 256, 64, True), (1, 0, [7, 1, 0, 300, 2, 3, 99, 513], 1304, 24, True),
            (2, 77, None, 40, 0, False), (2, 1500, None, 2560, 128, False)):
        inp = si.make_conv_inputs(batch, seqlen, x_dim, bc_dim, K, dtype, seed=4902,
                                  seq_lens=lens, history=hist)
        xbc = inp["xbc"].cuda()
        if lens is None:
            xbc = xbc.view(batch, seqlen, x_dim + 2 * bc_dim)
        args = (inp["weight"].cuda(), inp["bias"].cuda() if bias else None, x_dim, bc_dim,
                inp["history"].cuda() if hist else None, inp["cu_seqlens"])
        plain = ssd.conv1d_silu(xbc, *args)
        saved = ssd.conv1d_silu(xbc, *args, checkpoint=True)
        again = ssd.conv1d_silu(saved[4], *args)
        direct = ssd.conv1d_silu(saved[4].load(), *args)
        torch.cuda.synchronize()
        for k in range(4):
            assert torch.equal(saved[k], plain[k]), k
        for k in range(3):
            assert torch.equal(again[k], direct[k]), k
