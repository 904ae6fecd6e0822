"""The norm and rotation of keys and queries (ssd_bc_norm and its backward pass)
on the GPU against the fp64 oracle.

Bounds, per element (layer_helpers.check): C u times the magnitude of the terms,
u = 2^-24, and half a step of the output's type. Forward, C = 64: the squares'
sum over up to 8 channels of a lane and 5 levels of lanes is off by 16 u of itself,
halved by the root, whose hardware form and the products add 8; sine and cosine
of an angle reduced in 64 bits and rounded to fp32 add 2 pi / 2 half steps of a turn
(4 u) and 4 of their own; twice 4 for the two products of a turn and their sum; 64
holds them twice over. Backward, C = 256: h and dv at 64 each, the product's sum
over the head at 16 more, r at 16, all of it again in the difference. The weights'
gradients add up to 64 terms in a lane and 64 partial sums in turn: C = 512.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from layer_helpers import DT, check
from oracle.delta import bc_norm, bc_norm_backward

pytestmark = pytest.mark.gpu

CASES = {
    # name: (lead shape, B heads, C heads, dim, dtype, rotary, interleaved, unit, weights, start,
    #        positions over the last axis only)
    "one-token": ((1,), 1, 1, 128, "bf16", 0, False, True, False, 0, False),
    "one-token-rotated": ((1, 1), 8, 32, 128, "bf16", 64, False, False, True, 100000, False),
    "batch": ((3, 21), 2, 6, 128, "bf16", 128, False, True, True, 7, True),
    "batch-interleaved": ((3, 21), 2, 6, 128, "bf16", 128, True, True, True, 7, True),
    "dim-8": ((70,), 3, 1, 8, "bf16", 8, False, True, True, 0, False),
    "dim-16-interleaved": ((70,), 1, 5, 16, "fp32", 8, True, False, True, 3, False),
    "dim-48": ((33,), 5, 7, 48, "bf16", 32, False, False, True, 500, False),
    "dim-80-fp32": ((33,), 2, 2, 80, "fp32", 40, False, True, True, 500, False),
    "dim-200": ((9,), 4, 3, 200, "bf16", 200, True, True, False, 1, False),
    "dim-256-fp32": ((5, 31), 1, 1, 256, "fp32", 256, False, False, True, 0, False),
    "dim-256": ((5, 31), 3, 1, 256, "bf16", 8, False, False, True, 0, True),
    "far-positions": ((40,), 1, 2, 64, "fp32", 64, False, False, False, 2 ** 31 - 41, False),
    "no-rotation-fp32": ((300,), 6, 2, 128, "fp32", 0, False, False, True, 0, False),
    "many-tokens": ((9000,), 1, 3, 64, "bf16", 32, False, True, True, 0, False),
}


def _inputs(name, seed):
    lead, hb, hc, n, dtype, rot, inter, unit, weights, start, last = CASES[name]
    rng = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    d = {k: f(*lead, h, n).to(DT[dtype]) for k, h in (("B", hb), ("C", hc), ("dB", hb), ("dC", hc))}
    for side in "BC":
        d[side + "_weight"] = 1 + 0.3 * f(n) if weights else None
    kw = dict(eps=1e-6, unit=unit, interleaved=inter)
    if rot:
        shape = lead[-1:] if last else lead
        d["positions"] = (start + torch.arange(int(np.prod(shape)))).to(torch.int32).reshape(shape)
        d["freqs"] = torch.from_numpy((10000.0 ** -(np.arange(rot // 2) / (rot // 2)))
                                      .astype(np.float32))
    else:
        d["positions"] = d["freqs"] = None
    return d, kw


def _cuda(d):
    return {k: v if v is None else v.cuda() for k, v in d.items()}


def _forward(t, kw, **more):
    return ssd.bc_norm(t["B"], t["C"], t["B_weight"], t["C_weight"], t["positions"], t["freqs"],
                       **kw, **more)


def _backward(t, kw, **more):
    return ssd.bc_norm_backward(t["dB"], t["dC"], t["B"], t["C"], t["B_weight"], t["C_weight"],
                                t["positions"], t["freqs"], **kw, **more)


def _tokens(v):
    return v.reshape((-1,) + v.shape[-2:])


def _check_forward(got, d, kw, dtype):
    for side, o in zip("BC", got):
        want, size = bc_norm(_tokens(d[side]), d[side + "_weight"], d["positions"], d["freqs"], **kw)
        check(side + "_out", _tokens(o), want, size, dtype, 64)


def _check_backward(g, d, kw, dtype):
    for side in "BC":
        w = d[side + "_weight"]
        (dx, dw), (xs, ws) = bc_norm_backward(_tokens(d["d" + side]), _tokens(d[side]), w,
                                              d["positions"], d["freqs"], **kw)
        check("d" + side, _tokens(g["d" + side]), dx, xs, dtype, 256)
        assert (g["d%s_weight" % side] is None) == (w is None)
        if w is not None:
            check("d%s_weight" % side, g["d%s_weight" % side], dw, ws, "fp32", 512)


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name):
    d, kw = _inputs(name, 100 + sorted(CASES).index(name))
    print("[gpu] bc norm %s" % name, flush=True)
    _check_forward(_forward(_cuda(d), kw), d, kw, CASES[name][4])


@pytest.mark.parametrize("name", sorted(CASES))
def test_backward(name):
    d, kw = _inputs(name, 200 + sorted(CASES).index(name))
    print("[gpu] bc norm backward %s" % name, flush=True)
    _check_backward(_backward(_cuda(d), kw), d, kw, CASES[name][4])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zero_and_extreme_rows(dtype):
    """A row of zeros stays zero (eps > 0) and its gradient finite; large and small
    values do not overflow where their squares' sum does not."""
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((4, 2, 64)).astype(np.float32))
    x[1], x[2], x[3] = 0, x[2] * 1e15, x[3] * 1e-15
    x = x.to(DT[dtype])
    d = dict(B=x, C=x.flip(0), dB=torch.ones_like(x), dC=torch.ones_like(x), B_weight=None,
             C_weight=None, positions=None, freqs=None)
    kw = dict(eps=1e-12, unit=True, interleaved=False)
    print("[gpu] bc norm of extreme rows %s" % dtype, flush=True)
    got = _forward(_cuda(d), kw)
    assert not got[0][1].any() and not got[1][2].any()
    _check_forward(got, d, kw, dtype)
    _check_backward(_backward(_cuda(d), kw), d, kw, dtype)


def test_gradients_are_differences():
    """fp32 gradients against central differences of the fp32 forward call in random
    directions: step 2^-6 (truncation 2^-12 / 6 of a third derivative of the
    gradient's size over a head's scale), rounding 2^-24 * 2^6 of the loss' terms' norm."""
    d, kw = _inputs("dim-80-fp32", 6)
    kw["eps"] = 0.5
    t = _cuda(d)
    print("[gpu] bc norm differences", flush=True)
    g = _backward(t, kw)

    def loss(**more):
        b, c = _forward(dict(t, **more), kw)
        return float((b.double() * t["dB"].double()).sum() + (c.double() * t["dC"].double()).sum())

    rng = torch.Generator().manual_seed(1)
    step = 2.0 ** -6
    for k in ("B", "C", "B_weight", "C_weight"):
        v = torch.randn(t[k].shape, generator=rng).cuda()
        v /= v.norm()
        got = float((g["d" + k].double() * v.double()).sum())
        want = (loss(**{k: t[k] + step * v}) - loss(**{k: t[k] - step * v})) / (2 * step)
        assert abs(got - want) <= 1e-3 * float(g["d" + k].double().norm()), (k, got, want)


@pytest.mark.parametrize("name", ["batch", "dim-16-interleaved", "dim-256"])
def test_slices_and_outputs(name):
    """B and C side by side in wider rows, as one projection gives them, and outputs
    into such rows: the same bits, and nothing beside them is written."""
    lead, hb, hc, n, dtype = CASES[name][:5]
    d, kw = _inputs(name, 300)
    t = _cuda(d)
    want, gw = _forward(t, kw), _backward(t, kw)
    w = (hb + hc) * n

    def pair():
        wide = torch.full(lead + (w + 16,), 7.0, device="cuda", dtype=DT[dtype])
        return wide, wide[..., 8:8 + hb * n].unflatten(-1, (hb, n)), \
            wide[..., 8 + hb * n:8 + w].unflatten(-1, (hc, n))

    s = dict(t)
    for a, b in (("B", "C"), ("dB", "dC")):
        _, s[a], s[b] = pair()
        s[a].copy_(t[a])
        s[b].copy_(t[b])
    print("[gpu] bc norm slices %s" % name, flush=True)
    for f, want2, keys in ((_forward, want, ("B_out", "C_out")),
                           (_backward, (gw["dB"], gw["dC"]), ("dB", "dC"))):
        wide, o0, o1 = pair()
        got = f(s, kw, **dict(zip(keys, (o0, o1))))
        assert torch.equal(o0, want2[0]) and torch.equal(o1, want2[1])
        assert (wide[..., :8] == 7).all() and (wide[..., 8 + w:] == 7).all()
        if f is _backward:
            assert torch.equal(got["dB_weight"], gw["dB_weight"])
    # rows off 16 bytes and transposed heads are copied
    for k in ("B", "dC"):
        wide = torch.zeros(lead + (t[k].shape[-2] * n + 8,), device="cuda", dtype=DT[dtype])
        v = wide[..., 1:-7].unflatten(-1, t[k].shape[-2:])
        v.copy_(t[k])
        s[k] = v
    s["C"] = t["C"].transpose(-1, -2).contiguous().transpose(-1, -2)
    got = _forward(s, kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = _backward(s, kw)
    assert all(torch.equal(got[k], gw[k]) for k in gw)


def test_positions_of_both_types_and_without_tokens():
    d, kw = _inputs("batch", 400)
    t = _cuda(d)
    want = _forward(t, kw)
    print("[gpu] bc norm positions", flush=True)
    full = t["positions"].expand(3, 21)
    for p in (t["positions"].long(), full, full.contiguous().long()):
        got = _forward(dict(t, positions=p), kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e = {k: v if k in ("freqs", "B_weight", "C_weight") else v[:0] for k, v in t.items()
         if k != "positions"}
    e["positions"] = t["positions"]
    assert _forward(e, kw)[0].shape == (0, 21, 2, 128)
    g = _backward(e, kw)
    assert g["dB"].numel() == 0 and not g["dB_weight"].any() and not g["dC_weight"].any()


def test_rows_past_32_bits():
    """Rows whose last elements lie 2^31 elements and more behind the first."""
    tokens, row = 70000, 32768
    wide = torch.empty(tokens, row, device="cuda", dtype=torch.bfloat16)
    B, C = wide[:, :256].unflatten(1, (2, 128)), wide[:, 512:640].unflatten(1, (1, 128))
    B.normal_()
    C.normal_()
    assert (tokens - 1) * row > 1 << 31
    kw = dict(eps=1e-6, unit=True)
    print("[gpu] bc norm far rows", flush=True)
    got = ssd.bc_norm(B, C, **kw)
    want = ssd.bc_norm(B[-9:].contiguous(), C[-9:].contiguous(), **kw)
    assert torch.equal(got[0][-9:], want[0]) and torch.equal(got[1][-9:], want[1])
    out = wide[:, 1024:1280].unflatten(1, (2, 128))
    ssd.bc_norm(B, C, B_out=out, **kw)
    assert torch.equal(out, got[0])


def test_captured_on_two_streams():
    """Two graphs of forward and backward, replayed in turn on new inputs with eager
    work between; and eager calls on two streams."""
    name = "many-tokens"
    d = [_inputs(name, 500 + i) for i in range(3)]
    new, kw = [_cuda(v) for v, _ in d], d[0][1]

    def work(t, **more):
        g = _backward(t, kw, **more)
        return [*_forward(t, kw, **more), *(g[k] for k in g)]

    want = [work(t) for t in new]
    torch.cuda.synchronize()
    print("[gpu] bc norm captured", flush=True)
    graphs = []
    for _ in range(2):
        t = {k: v.clone() for k, v in new[0].items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = work(t)
        graphs.append((graph, t, out))
    for r in range(6):
        graph, t, out = graphs[r % 2]
        for k in t:
            t[k].copy_(new[r % 3][k])
        graph.replay()
        again = work(new[r % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[r % 3])), r
        assert all(torch.equal(a, b) for a, b in zip(again, want[r % 3])), r
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [work(new[i % 2], stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 2]))
