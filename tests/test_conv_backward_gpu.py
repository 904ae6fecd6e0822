"""The convolution front's backward pass (ssd_conv1d_silu_backward) on the GPU
against the fp64 oracle; bounds in layer_helpers."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
import ssd_inputs as si
from layer_helpers import check
from oracle.checkpoint import kept
from oracle.conv import dense_bounds, varlen_bounds
from oracle.conv_backward import conv_backward

pytestmark = pytest.mark.gpu

CASES = {
    # name: (batch, seqlen, seq_lens, x_dim, bc_dim, K, dtype, history, dhistory_out, lead, pad)
    "bf16-K4-dense-hist": (2, 300, None, 128, 32, 4, "bf16", True, True, 0, 0),
    "fp32-K4-dense": (3, 65, None, 64, 16, 4, "fp32", False, False, 0, 0),
    "bf16-K3-packed-short-empty": (1, 0, [1, 0, 37, 2, 100, 0, 64, 3], 64, 16, 3, "bf16", True,
                                   True, 0, 0),
    "bf16-K2-packed-empty-tail": (1, 0, [5, 40, 0, 0], 32, 8, 2, "bf16", True, False, 0, 0),
    "fp32-K3-slice-of-wider-rows": (2, 50, None, 64, 16, 3, "fp32", True, True, 64, 32),
    "bf16-K4-packed-slice": (1, 0, [33, 31, 64, 1], 256, 64, 4, "bf16", False, True, 128, 64),
    "fp32-K4-tile-edges": (1, 0, [61, 62, 60, 58, 59, 122, 123, 121, 0, 64, 183], 24, 8, 4,
                           "fp32", True, True, 0, 0),
    "bf16-K4-one-token": (5, 1, None, 64, 16, 4, "bf16", True, True, 0, 0),
    "fp32-K4-two-tokens": (4, 2, None, 40, 8, 4, "fp32", True, True, 0, 0),
    "bf16-K4-no-x-part": (2, 70, None, 0, 16, 4, "bf16", True, False, 0, 0),
    "fp32-K2-only-x": (1, 130, None, 72, 0, 2, "fp32", False, False, 0, 0),
    "bf16-K4-many-short": (1, 0, [3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 0, 8] * 20, 64, 8, 4, "bf16",
                           True, True, 0, 0),
    "bf16-K4-more-than-64-lanes": (1, 400, None, 1032, 24, 4, "bf16", False, False, 0, 0),
}


def _case(name):
    batch, seqlen, lens, x_dim, bc_dim, K, dtype, hist, dho, lead, pad = CASES[name]
    seed = 4500 + sorted(CASES).index(name)
    inp = si.make_conv_inputs(batch, seqlen, x_dim, bc_dim, K, dtype, seed=seed, seq_lens=lens,
                              history=hist, lead_cols=lead, pad_cols=pad)
    g = torch.Generator().manual_seed(seed)
    T, ch = inp["T"], x_dim + 2 * bc_dim
    dt = inp["xbc"].dtype
    d = torch.randn(T, ch, generator=g).to(dt)
    nseq = inp["num_seqs"] or inp["batch"]
    dh = torch.randn(nseq, K - 1, ch, generator=g).to(dt) if dho else None
    bounds = dense_bounds(batch, seqlen) if lens is None else varlen_bounds(inp["cu_seqlens"].tolist())
    return inp, d, dh, bounds, (x_dim, bc_dim, lens, lead, dtype)


def _gpu(inp, d, dh, meta, xbc=None, **kw):
    x_dim, bc_dim, lens, lead, _ = meta
    ch = x_dim + 2 * bc_dim
    shape = (lambda t: t) if lens is not None else \
        (lambda t: t.view(inp["batch"], inp["seqlen"], t.shape[-1]))
    if xbc is None:
        xbc = shape(inp["xbc_full"].cuda()[:, lead:lead + ch])
    dx, dB, dC = (shape(t.contiguous().cuda()) for t in d.split([x_dim, bc_dim, bc_dim], 1))
    cuda = lambda t: None if t is None else t.cuda()
    return ssd.conv1d_silu_backward(xbc, inp["weight"].cuda(), inp["bias"].cuda(), dx, dB, dC,
                                    cuda(inp["history"]), inp["cu_seqlens"],
                                    dhistory_out=cuda(dh), **kw)


def _compare(got, want, size, dtype, hist):
    for k in ("dxbc", "dweight", "dbias", "dhistory"):
        if k == "dhistory" and not hist:
            assert got[k] is None
            continue
        check(k, got[k], want[k], size[k], "fp32" if k in ("dweight", "dbias") else dtype, 160)


@pytest.mark.parametrize("name", sorted(CASES))
def test_conv_backward(name):
    inp, d, dh, bounds, meta = _case(name)
    print("[gpu] conv backward %s" % name, flush=True)
    got = _gpu(inp, d, dh, meta)
    torch.cuda.synchronize()
    want, size = conv_backward(inp["xbc"], inp["weight"], inp["bias"], bounds, d, inp["history"], dh)
    _compare(got, want, size, meta[4], inp["history"] is not None)


@pytest.mark.parametrize("name", sorted(CASES))
def test_conv_backward_from_checkpoint(name):
    """From an 8-bit checkpoint: the gradients at the values it holds."""
    inp, d, dh, bounds, meta = _case(name)
    print("[gpu] conv backward from 8 bits %s" % name, flush=True)
    xbc = inp["xbc"].contiguous().cuda()
    if meta[2] is None:
        xbc = xbc.view(inp["batch"], inp["seqlen"], -1)
    got = _gpu(inp, d, dh, meta, xbc=ssd.checkpoint_save(xbc))
    torch.cuda.synchronize()
    want, size = conv_backward(kept(inp["xbc"]), inp["weight"], inp["bias"], bounds, d,
                               inp["history"], dh)
    _compare(got, want, size, meta[4], inp["history"] is not None)


def test_conv_backward_zero_tokens():
    """Rows without tokens: zero sums, and the history's gradient is that of
    the history that passed through."""
    ch, K = 48, 3
    hist = torch.randn(4, K - 1, ch, device="cuda").to(torch.bfloat16)
    dh = torch.randn(4, K - 1, ch, device="cuda").to(torch.bfloat16)
    w, b = torch.randn(ch, K, device="cuda"), torch.randn(ch, device="cuda")
    e = lambda n: torch.empty(4, 0, n, dtype=torch.bfloat16, device="cuda")
    print("[gpu] conv backward zero tokens", flush=True)
    g = ssd.conv1d_silu_backward(e(ch), w, b, e(32), e(8), e(8), hist, dhistory_out=dh)
    g0 = ssd.conv1d_silu_backward(e(ch), w, b, e(32), e(8), e(8), hist)
    torch.cuda.synchronize()
    assert torch.equal(g["dhistory"], dh) and torch.count_nonzero(g0["dhistory"]) == 0
    assert torch.count_nonzero(g["dweight"]) == 0 and torch.count_nonzero(g["dbias"]) == 0
    e0 = lambda n: torch.empty(0, 5, n, dtype=torch.bfloat16, device="cuda")
    g = ssd.conv1d_silu_backward(e0(ch), w, None, e0(32), e0(8), e0(8))
    torch.cuda.synchronize()
    assert torch.count_nonzero(g["dweight"]) == 0 and g["dxbc"].shape == (0, 5, ch)


def test_conv_backward_into_a_slice():
    """dxbc as a slice of wider rows leaves the columns beside it; equal calls
    give equal bits; the gradients come in the shapes ssd.backward returns."""
    inp, d, dh, _, meta = _case("bf16-K4-dense-hist")
    print("[gpu] conv backward into a slice", flush=True)
    want = _gpu(inp, d, dh, meta)
    ch = 192
    wide = torch.full((2, 300, ch + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    got = _gpu(inp, d, dh, meta, dxbc=wide[:, :, 32:32 + ch])
    dx, dB, dC = (t.contiguous().cuda() for t in d.split([128, 32, 32], 1))
    heads = ssd.conv1d_silu_backward(
        inp["xbc"].cuda().view(2, 300, ch), inp["weight"].cuda(), inp["bias"].cuda(),
        dx.view(2, 300, 2, 64), dB.view(2, 300, 1, 32), dC.view(2, 300, 2, 16),
        inp["history"].cuda(), dhistory_out=dh.cuda())
    # gradients and histories that must be copied first: strided, or 2 bytes off
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
    odd = ssd.conv1d_silu_backward(
        off(inp["xbc"].cuda().view(2, 300, ch)), inp["weight"].cuda(), inp["bias"].cuda(),
        off(dx.view(2, 300, 128)), dB.view(2, 300, 32).transpose(0, 1).contiguous().transpose(0, 1),
        off(dC.view(2, 300, 32)), off(inp["history"].cuda()), dhistory_out=off(dh.cuda()))
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
        assert torch.equal(heads[k], want[k]), k
        assert torch.equal(odd[k], want[k]), k
    assert (wide[:, :, :32] == 3).all() and (wide[:, :, 32 + ch:] == 3).all()


def test_conv_backward_splits_like_the_forward():
    """A sequence cut in two, the second part's dhistory given to the first
    part as dhistory_out, has the gradients of the whole (fp32)."""
    inp, d, _, bounds, meta = _case("fp32-K4-dense")
    print("[gpu] conv backward in two parts", flush=True)
    whole = _gpu(inp, d, None, meta)
    w, b = inp["weight"].cuda(), inp["bias"].cuda()
    xbc, dd = inp["xbc"].cuda().view(3, 65, 96), d.cuda().view(3, 65, 96)
    for cut in (1, 2, 40, 64):
        parts = lambda a, e: [t.contiguous() for t in dd[:, a:e].split([64, 16, 16], 2)]
        zero = torch.zeros(3, 3, 96, device="cuda")
        hist = ssd.conv1d_silu(xbc[:, :cut].contiguous(), w, b, 64, 16, zero)[3]
        g2 = ssd.conv1d_silu_backward(xbc[:, cut:].contiguous(), w, b, *parts(cut, 65), hist)
        g1 = ssd.conv1d_silu_backward(xbc[:, :cut].contiguous(), w, b, *parts(0, cut), zero,
                                      dhistory_out=g2["dhistory"])
        torch.cuda.synchronize()
        dxbc = torch.cat([g1["dxbc"], g2["dxbc"]], 1)
        # the same terms in another order: 8 roundings of sums of a few units
        assert torch.allclose(dxbc, whole["dxbc"], rtol=0, atol=8e-6), cut
        for k in ("dweight", "dbias"):
            assert torch.allclose(g1[k] + g2[k], whole[k], rtol=0, atol=2e-4), (cut, k)


def test_conv_backward_full_workload_sampled():
    """The 2.7B-shaped front (batch 8, 2048 tokens, 5376 channels, bf16);
    sampled channels against the oracle (channels are independent)."""
    x_dim, bc_dim, K = 5120, 128, 4
    inp = si.make_conv_inputs(8, 2048, x_dim, bc_dim, K, "bf16", seed=4700)
    ch = x_dim + 2 * bc_dim
    d = torch.randn(8 * 2048, ch, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    print("[gpu] conv backward full workload", flush=True)
    got = _gpu(inp, d, None, (x_dim, bc_dim, None, 0, "bf16"))
    torch.cuda.synchronize()
    sel = torch.as_tensor([0, 7, 511, 512, 2600, 5119, 5120, 5247, 5248, 5375])
    want, size = conv_backward(inp["xbc"][:, sel], inp["weight"][sel], inp["bias"][sel],
                               dense_bounds(8, 2048), d[:, sel])
    pick = lambda k: got[k].reshape(-1, ch)[:, sel.cuda()] if k == "dxbc" else got[k][sel.cuda()]
    for k in ("dxbc", "dweight", "dbias"):
        check(k, pick(k), want[k], size[k], "bf16" if k == "dxbc" else "fp32", 160)


@pytest.mark.parametrize("K,dtype,lens,keep", [
    (4, torch.bfloat16, None, False), (4, torch.bfloat16, [1201, 0, 3, 36, 1260], True),
    (3, torch.float32, [1, 2499], False), (2, torch.float32, None, True)])
def test_conv_backward_many_channels_sampled(K, dtype, lens, keep):
    """65,536 channels; sampled channels against the oracle (channels are
    independent)."""
    x_dim, bc_dim, T = 65024, 256, 2500
    ch, dev = x_dim + 2 * bc_dim, "cuda"
    name = "bf16" if dtype == torch.bfloat16 else "fp32"
    g = torch.Generator(device=dev).manual_seed(4800 + K)
    rand = lambda *shape, dt=dtype: torch.randn(shape, device=dev, generator=g,
                                                dtype=torch.float32).to(dt)
    nseq = 2 if lens is None else len(lens)
    u, w, b = rand(T, ch), rand(ch, K, dt=torch.float32), rand(ch, dt=torch.float32)
    grads = [rand(T, n) for n in (x_dim, bc_dim, bc_dim)]
    hist, dh = rand(nseq, K - 1, ch), rand(nseq, K - 1, ch)
    cu = None if lens is None else torch.tensor(np.cumsum([0] + lens), dtype=torch.int32)
    lead = (lambda t: t.view(2, T // 2, -1)) if lens is None else (lambda t: t)
    xbc = ssd.checkpoint_save(lead(u)) if keep else lead(u)
    print("[gpu] conv backward many channels", K, dtype, lens, keep, flush=True)
    got = ssd.conv1d_silu_backward(xbc, w, b, *(lead(t) for t in grads), hist, cu,
                                   dhistory_out=dh)
    torch.cuda.synchronize()
    sel = torch.as_tensor([0, 5, 255, 256, 32767, 65023, 65024, 65279, 65280, 65535], device=dev)
    seen = xbc.load().reshape(T, ch) if keep else u
    cpu = lambda t: t.cpu()
    bounds = dense_bounds(2, T // 2) if lens is None else varlen_bounds(cu.tolist())
    want, size = conv_backward(cpu(seen[:, sel]), cpu(w[sel]), cpu(b[sel]), bounds,
                               cpu(torch.cat(grads, 1)[:, sel]), cpu(hist[:, :, sel]),
                               cpu(dh[:, :, sel]))
    pick = dict(dxbc=got["dxbc"].reshape(T, ch)[:, sel], dweight=got["dweight"][sel],
                dbias=got["dbias"][sel], dhistory=got["dhistory"][:, :, sel])
    for k, v in pick.items():
        check(k, v, want[k], size[k], name if k in ("dxbc", "dhistory") else "fp32", 160)


def test_conv_backward_offsets_that_are_no_partition():
    """Device offsets that are not checked (descending, negative, past the end)
    stay inside the tensors: nothing but the outputs changes."""
    ch, K, T = 96, 4, 200
    xbc = torch.randn(T, ch, device="cuda").to(torch.bfloat16)
    w = torch.randn(ch, K, device="cuda")
    dx, dB, dC = (torch.randn(T, n, device="cuda").to(torch.bfloat16) for n in (64, 16, 16))
    wide = torch.full((T + 2, ch), 5.0, dtype=torch.bfloat16, device="cuda")
    print("[gpu] conv backward with bad offsets", flush=True)
    for cu in ([0, 300, 200], [0, -7, 200], [0, 150, 20, 200], [2 ** 31 - 1, 0, -2 ** 31, 200]):
        ssd.conv1d_silu_backward(xbc, w, None, dx, dB, dC, None,
                                 torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                 dxbc=wide[1:-1], check_cu_seqlens=False)
        torch.cuda.synchronize()
        assert (wide[0] == 5).all() and (wide[-1] == 5).all()
    with pytest.raises(ValueError, match="cu_seqlens"):
        ssd.conv1d_silu_backward(xbc, w, None, dx, dB, dC, None,
                                 torch.tensor([0, 300, 200], dtype=torch.int32, device="cuda"))


def test_conv_backward_of_the_packed_layer():
    """Packed input, the layer's gradients as ssd.backward returns them (a batch
    axis of 1): what their flattened form gives, from xbc and from 8 bits."""
    H, P, G, N, K, lens = 4, 64, 1, 64, 4, [5, 0, 90, 1, 31]
    X, BC, T = H * P, G * N, sum(lens)
    inp = si.make_conv_inputs(1, 0, X, BC, K, "bf16", seed=4950, seq_lens=lens)
    xbc, w, b, cu = (inp[k].cuda() for k in ("xbc", "weight", "bias", "cu_seqlens"))
    g = torch.Generator().manual_seed(4951)
    dt = torch.rand(1, T, H, generator=g).to(torch.bfloat16).cuda()
    A, dy = -torch.rand(H, generator=g).cuda(), torch.randn(1, T, H, P, generator=g)
    print("[gpu] conv backward of the packed layer", flush=True)
    x, B, C, _, kept_ = ssd.conv1d_silu(xbc, w, b, X, BC, None, cu, checkpoint=True)
    gs = ssd.backward(x.view(1, T, H, P), dt, A, B.view(1, T, G, N), C.view(1, T, G, N), None, None,
                      dy.to(torch.bfloat16).cuda(), cu_seqlens=cu)
    assert gs["dx"].shape == (1, T, H, P) and gs["dB"].shape == (1, T, G, N)
    flat = [gs[k].reshape(T, -1) for k in ("dx", "dB", "dC")]
    for src in (xbc, kept_):
        got = ssd.conv1d_silu_backward(src, w, b, gs["dx"], gs["dB"], gs["dC"], None, cu)
        want = ssd.conv1d_silu_backward(src, w, b, *flat, None, cu)
        torch.cuda.synchronize()
        for k in ("dxbc", "dweight", "dbias"):
            assert got[k].shape == want[k].shape and torch.equal(got[k], want[k]), k
