"""The gated delta rule as a layer uses it: convolution front, norm and rotation of
the keys and queries, the rule, and the gated norm behind it; forwards and
backwards, and decoding token by token after a prefill. Against the fp64 oracles
run one after the other.

fp32: each of the four operators is within 80 u (u = 2^-24) of its own inputs'
result in norm, and a later one carries an earlier one's error on by at most 4
(the norms' slope at these inputs): (1 + 4 + 16 + 64) * 80 u = 4e-4 holds the chain,
and the chain backwards once more: 8e-4.
bf16: each hands on values rounded by 2^-8 (2^-8 / sqrt(3) in the root mean square),
the rule's own 2.6 * 2^-8 among them; eight roundings on the way back, carried on by
at most 2: sqrt(8) * 2 * 2.6 * 2^-8 = 5.7e-2.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import mamba_ssd_sequence_fwd_amd as ssd
from delta_helpers import DT
from oracle import _np
from oracle.conv import conv_front, dense_bounds, varlen_bounds
from oracle.conv_backward import conv_backward
from oracle.delta import bc_norm, bc_norm_backward, delta_backward, delta_rule
from oracle.norm import norm, norm_backward

pytestmark = pytest.mark.gpu

H, P, G, N, K, ROT = 4, 32, 2, 64, 4, 32
XD, BD = H * P, G * N
NORM = dict(eps=1e-6, unit=True)
FREQS = (100.0 ** -(np.arange(ROT // 2) / (ROT // 2))).astype(np.float32)
BOUND = {"fp32": (4e-4, 8e-4), "bf16": (2.9e-2, 5.7e-2)}


def _layer(seed, tokens, dtype):
    rng = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=rng)
    w = dict(conv=0.5 * r(XD + 2 * BD, K), bias=0.1 * r(XD + 2 * BD), bw=1 + 0.1 * r(N),
             cw=1 + 0.1 * r(N), nw=1 + 0.1 * r(XD))
    a = dict(xbc=r(tokens, XD + 2 * BD), z=r(tokens, XD), beta=torch.sigmoid(r(tokens, H)),
             g=-0.3 * torch.nn.functional.softplus(r(tokens, H)), dout=r(tokens, XD))
    return w, {k: v.to(DT[dtype]) for k, v in a.items()}


def _err(got, want):
    g = got.detach().double().cpu().numpy().reshape(want.shape)
    return np.linalg.norm(g - want) / np.linalg.norm(want)


def _run(w, a, lead, cu, positions, history=None, h0=None):
    """The chain on the GPU: (out, history, state, what the way back needs)."""
    v = lambda t: t.reshape(lead + t.shape[1:])
    xbc = a["xbc"] if cu is not None else v(a["xbc"])
    x, B, C, hist = ssd.conv1d_silu(xbc, w["conv"], w["bias"], XD, BD, history, cu)
    x = x.reshape(lead + (H, P))
    B, C = B.reshape(lead + (G, N)), C.reshape(lead + (G, N))
    k, q = ssd.bc_norm(B, C, w["bw"], w["cw"], positions, w["freqs"], **NORM)
    y, state = ssd.delta_forward(x, v(a["g"]), v(a["beta"]), k, q, h0, cu)
    yf = y.reshape(-1, XD)
    out = ssd.group_norm_silu(yf, w["nw"], None, a["z"], groups=1, eps=1e-5)
    return out, hist, state, dict(x=x, B=B, C=C, k=k, q=q, y=yf)


def _oracle(w, a, bounds, lens, positions):
    x, B, C, _ = conv_front(a["xbc"], w["conv"], w["bias"], bounds, XD, BD, None)
    T = x.shape[0]
    x, B, C = x.reshape(T, H, P), B.reshape(T, G, N), C.reshape(T, G, N)
    k, _ = bc_norm(B, w["bw"], positions, FREQS, **NORM)
    q, _ = bc_norm(C, w["cw"], positions, FREQS, **NORM)
    y, state = delta_rule(x, a["g"], a["beta"], k, q, None, lens)
    y = y.reshape(T, XD)
    out, _ = norm(y, _np(a["z"]), _np(w["nw"]), None, 1, 1e-5, False, "first")
    return out, state, dict(x=x, B=B, C=C, k=k, q=q, y=y)


def _dev(d):
    d = {k: v.cuda() for k, v in d.items()}
    return d


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_training_step(dtype, packed):
    lens = [70, 0, 1, 129] if packed else [100, 100]
    T = sum(lens)
    w, a = _layer(11, T, dtype)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32) if packed else None
    lead = (1, T) if packed else (2, 100)
    positions = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    t, s = _dev(w), _dev(a)
    t["freqs"] = torch.from_numpy(FREQS).cuda()
    pos = positions.reshape(lead).cuda()
    print("[gpu] delta layer %s packed=%s" % (dtype, packed), flush=True)
    out, _, state, m = _run(t, s, lead, cu, pos)
    bounds = varlen_bounds(cu.tolist()) if packed else dense_bounds(2, 100)
    want, hw, n = _oracle(w, a, bounds, lens, positions)
    assert _err(out, want) <= BOUND[dtype][0], _err(out, want)
    assert _err(state, hw) <= BOUND[dtype][0]

    # and back
    v = lambda x: x.reshape(lead + x.shape[1:])
    gn = ssd.group_norm_silu_backward(s["dout"], m["y"], t["nw"], None, s["z"], groups=1, eps=1e-5)
    gd = ssd.delta_backward(m["x"], v(s["g"]), v(s["beta"]), m["k"], m["q"], None,
                            gn["dx"].reshape(m["x"].shape), None, cu)
    gb = ssd.bc_norm_backward(gd["dB"], gd["dC"], m["B"], m["C"], t["bw"], t["cw"], pos,
                              t["freqs"], **NORM)
    flat = (lambda x: x.reshape(T, -1)) if packed else (lambda x: x.reshape(2, 100, -1))
    gc = ssd.conv1d_silu_backward(flat(s["xbc"]), t["conv"], t["bias"], flat(gd["dx"]),
                                  flat(gb["dB"]), flat(gb["dC"]), cu_seqlens=cu)
    torch.cuda.synchronize()
    on, _ = norm_backward(_np(a["dout"]), n["y"], _np(a["z"]), _np(w["nw"]), None, 1, 1e-5, False,
                          "first")
    od = delta_backward(n["x"], a["g"], a["beta"], n["k"], n["q"], None, lens,
                        on["dx"].reshape(T, H, P))
    (oB, obw), _ = bc_norm_backward(od["dB"], n["B"], w["bw"], positions, FREQS, **NORM)
    (oC, ocw), _ = bc_norm_backward(od["dC"], n["C"], w["cw"], positions, FREQS, **NORM)
    got = dict(dz=(gn["dz"], on["dz"]), dnorm=(gn["dweight"], on["dweight"]),
               dg=(gd["dg"], od["dg"]), dbeta=(gd["dbeta"], od["dbeta"]),
               dB_weight=(gb["dB_weight"], obw), dC_weight=(gb["dC_weight"], ocw),
               dx=(gd["dx"], od["dx"]), dB=(gb["dB"], oB), dC=(gb["dC"], oC))
    oc, _ = conv_backward(a["xbc"], w["conv"], w["bias"], bounds,
                          np.concatenate([v.reshape(T, -1) for v in (od["dx"], oB, oC)], axis=1))
    for k in ("dxbc", "dweight", "dbias"):
        got[k] = (gc[k], oc[k])
    for k, (g, o) in got.items():
        assert _err(g, o) <= BOUND[dtype][1], (k, _err(g, o))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_decoding_follows_the_prefill(dtype):
    """37 tokens at once, then 5 one by one with the front's history, the positions
    and the state carried on: the outputs of all 42 at once."""
    T, L, S = 42, 37, 3
    w, a = _layer(12, S * T, dtype)
    t, s = _dev(w), _dev(a)
    t["freqs"] = torch.from_numpy(FREQS).cuda()
    pos = torch.arange(T, device="cuda")
    part = lambda lo, hi: {k: v.reshape((S, T) + v.shape[1:])[:, lo:hi].reshape(
        (-1,) + v.shape[1:]) for k, v in s.items()}
    print("[gpu] delta layer decodes %s" % dtype, flush=True)
    whole = _run(t, s, (S, T), None, pos)
    out, hist, state, _ = _run(t, part(0, L), (S, L), None, pos[:L])
    outs = [out.reshape(S, L, XD)]
    for i in range(L, T):
        one = part(i, i + 1)
        x, B, C, hist = ssd.conv1d_silu(one["xbc"].reshape(S, 1, -1), t["conv"], t["bias"], XD, BD,
                                        hist)
        k, q = ssd.bc_norm(B.reshape(S, G, N), C.reshape(S, G, N), t["bw"], t["cw"],
                           pos[i:i + 1].expand(S), t["freqs"], **NORM)
        y = ssd.delta_step(x.reshape(S, H, P), one["g"], one["beta"], k, q, state)
        outs.append(ssd.group_norm_silu(y.reshape(S, XD), t["nw"], None, one["z"], groups=1,
                                        eps=1e-5).reshape(S, 1, XD))
    torch.cuda.synchronize()
    got = torch.cat(outs, 1).reshape(S * T, XD)
    want, hw, _ = _oracle(w, a, dense_bounds(S, T), [T] * S,
                          np.tile(np.arange(T), S))
    assert _err(got, want) <= BOUND[dtype][0]
    assert _err(whole[0], want) <= BOUND[dtype][0]
    assert _err(state, hw) <= BOUND[dtype][0] and _err(whole[2], hw) <= BOUND[dtype][0]
