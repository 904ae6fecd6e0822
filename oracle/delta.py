"""fp64 oracle of the gated delta rule, its gradients, and the norm and rotation
of its keys and queries.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``. Token by token; per head,
with the state h (P, N), the value x, the key k = B and the query q = C:

    h = e^g h;  e = beta (x - h k);  h = h + e k^T;  y = h q

and the same walked backwards.
"""
from __future__ import annotations

import numpy as np

from oracle import _np, seq_layout


def _heads(v, H):
    """(T, G, N) -> (T, H, N): a group's row for each of its heads."""
    return np.repeat(v, H // v.shape[1], axis=1)


def delta_rule(x, g, beta, B, C, h0=None, seq_lens=None):
    """x (T, H, P); g, beta (T, H); B, C (T, G, N); h0 (S, H, P, N) or None.
    Returns (y, final state (S, H, P, N))."""
    x, g, beta, B, C = (_np(v) for v in (x, g, beta, B, C))
    T, H, P = x.shape
    N = B.shape[2]
    K, Q = _heads(B, H), _heads(C, H)
    starts, lens = seq_layout(T, seq_lens)
    y = np.zeros((T, H, P))
    hT = np.zeros((len(lens), H, P, N))
    for s, (a, L) in enumerate(zip(starts, lens)):
        h = np.zeros((H, P, N)) if h0 is None else _np(h0)[s].copy()
        for t in range(a, a + L):
            h *= np.exp(g[t])[:, None, None]
            e = beta[t][:, None] * (x[t] - (h @ K[t][:, :, None])[:, :, 0])
            h += e[:, :, None] * K[t][:, None, :]
            y[t] = (h @ Q[t][:, :, None])[:, :, 0]
        hT[s] = h
    return y, hT


def delta_backward(x, g, beta, B, C, h0, seq_lens, dy, dhT=None):
    """dict of dx, dg, dbeta, dB, dC, dinitial_state."""
    x, g, beta, B, C, dy = (_np(v) for v in (x, g, beta, B, C, dy))
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    K, Q = _heads(B, H), _heads(C, H)
    starts, lens = seq_layout(T, seq_lens)
    dx, dg, dbeta = np.zeros_like(x), np.zeros_like(g), np.zeros_like(g)
    dK, dQ = np.zeros((T, H, N)), np.zeros((T, H, N))
    dh0 = np.zeros((len(lens), H, P, N))
    column = lambda h, v: (h @ v[:, :, None])[:, :, 0]       # (H, P, N) (H, N) -> (H, P)
    row = lambda h, v: (v[:, None, :] @ h)[:, 0, :]          # (H, P, N) (H, P) -> (H, N)
    for s, (a, L) in enumerate(zip(starts, lens)):
        h = np.zeros((H, P, N)) if h0 is None else _np(h0)[s].copy()
        decayed, errors = [], []
        for t in range(a, a + L):
            h = h * np.exp(g[t])[:, None, None]
            e = beta[t][:, None] * (x[t] - column(h, K[t]))
            decayed.append(h)
            errors.append(e)
            h = h + e[:, :, None] * K[t][:, None, :]
        D = np.zeros((H, P, N)) if dhT is None else _np(dhT)[s].copy()
        for t in range(a + L - 1, a - 1, -1):
            d, e = decayed[t - a], errors[t - a]
            h = d + e[:, :, None] * K[t][:, None, :]
            D += dy[t][:, :, None] * Q[t][:, None, :]
            dQ[t] = row(h, dy[t])
            Dk = column(D, K[t])
            de = beta[t][:, None] * Dk
            dx[t] = de
            dbeta[t] = (Dk * (x[t] - column(d, K[t]))).sum(axis=1)
            dK[t] = row(D, e) - row(d, de)
            D -= de[:, :, None] * K[t][:, None, :]
            dg[t] = (D * d).sum(axis=(1, 2))
            D *= np.exp(g[t])[:, None, None]
        dh0[s] = D
    group = lambda v: v.reshape(T, G, H // G, N).sum(axis=2)
    return dict(dx=dx, dg=dg, dbeta=dbeta, dB=group(dK), dC=group(dQ), dinitial_state=dh0)


def _pairs(n, interleaved):
    return (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n),
                                                                         slice(n, 2 * n))


def _pair_sums(v, n, interleaved):
    """|v|, and |u| + |w| in both channels of each of the n pairs (u, w)."""
    i, j = _pairs(n, interleaved)
    size = np.abs(v)
    size[..., i] = size[..., j] = size[..., i] + size[..., j]
    return size


def _turned(v, angle, interleaved, back=False):
    """The first 2 * angle.shape[-1] channels of v (T, heads, N) turned in pairs."""
    n = angle.shape[1]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    if back:
        s = -s
    i, j = _pairs(n, interleaved)
    out = v.copy()
    out[..., i] = v[..., i] * c - v[..., j] * s
    out[..., j] = v[..., i] * s + v[..., j] * c
    return out


def _angles(T, positions, freqs):
    if freqs is None or len(freqs) == 0:
        return np.zeros((T, 0))
    p = np.resize(_np(positions).reshape(-1), T)
    return p[:, None] * _np(freqs)[None, :]


def bc_norm(x, weight=None, positions=None, freqs=None, *, eps, unit=False, interleaved=False):
    """One side: x (T, heads, N). Returns (out, size): size bounds the terms of out."""
    x = _np(x)
    w = np.ones(x.shape[2]) if weight is None else _np(weight)
    r = 1 / np.sqrt((x * x).sum(axis=2, keepdims=True) / (1 if unit else x.shape[2]) + eps)
    v = x * r * w
    angle = _angles(x.shape[0], positions, freqs)
    out = _turned(v, angle, interleaved)
    return out, _pair_sums(v, angle.shape[1], interleaved)


def bc_norm_backward(dout, x, weight=None, positions=None, freqs=None, *, eps, unit=False,
                     interleaved=False):
    """One side: (dx, dweight) and the magnitudes of their terms."""
    dout, x = _np(dout), _np(x)
    T, _, N = x.shape
    w = np.ones(N) if weight is None else _np(weight)
    n = 1 if unit else N
    r = 1 / np.sqrt((x * x).sum(axis=2, keepdims=True) / n + eps)
    h = x * r
    angle = _angles(T, positions, freqs)
    dv = _turned(dout, angle, interleaved, back=True)
    top = _pair_sums(dout, angle.shape[1], interleaved)
    dh = dv * w
    dx = r * (dh - h * (dh * h).sum(axis=2, keepdims=True) / n)
    size = r * (top * np.abs(w) + np.abs(h) * (top * np.abs(w * h)).sum(axis=2, keepdims=True) / n)
    return (dx, (dv * h).sum(axis=(0, 1))), (size, (top * np.abs(h)).sum(axis=(0, 1)))
