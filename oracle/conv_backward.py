"""fp64 oracle of the convolution front's backward pass.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``. For one sequence with
e = [history rows, inputs] and pre as in ``oracle/conv.py``:

    g[t]  = dout[t] * silu'(pre[t]),   silu'(v) = sig(v) (1 + v (1 - sig(v)))
    de[j] = sum_k weight[:, k] g[j - k] + dhistory_out[j - L] (j >= L)
    dweight[:, k] = sum_t g[t] e[t + k],  dbias = sum_t g[t]

written as scatters per tap (the transpose of the forward's gathers). Every
result comes with the sum of the magnitudes of its terms, for error bounds.
"""
from __future__ import annotations

import numpy as np
from scipy.special import expit

from oracle.conv import _f64


def dsilu(v):
    s = expit(v)
    return s * (1.0 + v * (1.0 - s))


def conv_backward(xbc, weight, bias, seq_bounds, dout, history=None, dhistory_out=None):
    """xbc, dout (T, ch); weight (ch, K); history, dhistory_out (S, K - 1, ch)
    or None. Returns (grads, sizes): dicts with dxbc, dweight, dbias,
    dhistory, and the sums of their terms' magnitudes."""
    xbc, weight, bias, dout, history, dhistory_out = (
        _f64(v) for v in (xbc, weight, bias, dout, history, dhistory_out))
    T, ch = xbc.shape
    K = weight.shape[1]
    S = len(seq_bounds)
    out = dict(dxbc=np.zeros((T, ch)), dweight=np.zeros((ch, K)), dbias=np.zeros(ch),
               dhistory=np.zeros((S, K - 1, ch)))
    size = {k: v.copy() for k, v in out.items()}
    for s, (a, b) in enumerate(seq_bounds):
        L = b - a
        h = np.zeros((K - 1, ch)) if history is None else history[s]
        e = np.concatenate([h, xbc[a:b]], axis=0)
        pre = np.zeros((L, ch)) if bias is None else np.repeat(bias[None], L, axis=0)
        for k in range(K):
            pre = pre + weight[None, :, k] * e[k:k + L]
        g = dout[a:b] * dsilu(pre)
        # terms of silu', and half of pre's (|silu''| <= 1/2)
        terms = sum(np.abs(weight[None, :, k] * e[k:k + L]) for k in range(K))
        sg = np.abs(dout[a:b]) * (expit(pre) * (1 + np.abs(pre)) + 0.5 * (1 + terms))
        de, se = np.zeros_like(e), np.zeros_like(e)
        for k in range(K):
            de[k:k + L] += weight[None, :, k] * g
            se[k:k + L] += np.abs(weight[None, :, k]) * sg
            out["dweight"][:, k] += (g * e[k:k + L]).sum(axis=0)
            size["dweight"][:, k] += (sg * np.abs(e[k:k + L])).sum(axis=0)
        if dhistory_out is not None:
            de[L:] += dhistory_out[s]
            se[L:] += np.abs(dhistory_out[s])
        out["dbias"] += g.sum(axis=0)
        size["dbias"] += sg.sum(axis=0)
        out["dhistory"][s], out["dxbc"][a:b] = de[:K - 1], de[K - 1:]
        size["dhistory"][s], size["dxbc"][a:b] = se[:K - 1], se[K - 1:]
    return out, size
