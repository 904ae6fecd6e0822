"""fp64 oracle of the group norm with SiLU behind the SSD layer.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``. Per token and group of
n consecutive channels, silu(v) = v sig(v):

    u = x silu(z) (gate "first") or x;  mu = mean(u) if center else 0
    r = (mean((u - mu)^2) + eps)^-1/2;  h = (u - mu) r;  v = h weight + bias
    out = v ("first"), v silu(z) ("last"), silu(v) ("none")

and its gradients. Results come with the magnitude of the terms they are made
of, for error bounds.
"""
from __future__ import annotations

import numpy as np
from scipy.special import expit

from oracle.conv import _f64
from oracle.conv_backward import dsilu


def _silu(v):
    return v * expit(v)


def _stats(x, z, groups, eps, center, gate):
    u = x * _silu(z) if gate == "first" else x
    T, C = u.shape
    g = u.reshape(T, groups, C // groups)
    mu = g.mean(axis=2, keepdims=True) if center else np.zeros((T, groups, 1))
    r = 1.0 / np.sqrt(((g - mu) ** 2).mean(axis=2, keepdims=True) + eps)
    h = ((g - mu) * r).reshape(T, C)
    top = ((np.abs(g).max(axis=2, keepdims=True) + np.abs(mu)) * r)     # of h's terms
    return u, np.broadcast_to(r, g.shape).reshape(T, C), h, \
        np.broadcast_to(top, g.shape).reshape(T, C)


def norm(x, z, weight, bias, groups, eps, center, gate):
    """(out, size): the output and the magnitude of its terms."""
    x, z, weight, bias = (_f64(v) for v in (x, z, weight, bias))
    C = x.shape[1]
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    _, _, h, top = _stats(x, z, groups, eps, center, gate)
    v, size = h * w + b, top * np.abs(w) + np.abs(b)
    if gate == "last":
        return v * _silu(z), size * np.abs(_silu(z))
    if gate == "none":
        return _silu(v), size * (np.abs(dsilu(v)) + np.abs(expit(v)))
    return v, size


def norm_backward(dout, x, z, weight, bias, groups, eps, center, gate):
    """(grads, sizes) with dx, dz (None without a gate), dweight, dbias."""
    dout, x, z, weight, bias = (_f64(v) for v in (dout, x, z, weight, bias))
    T, C = x.shape
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    u, r, h, top = _stats(x, z, groups, eps, center, gate)
    v, vsize = h * w + b, top * np.abs(w) + np.abs(b)
    dv, dvsize = dout, np.abs(dout)
    if gate == "last":
        dv, dvsize = dout * _silu(z), np.abs(dout * _silu(z))
    elif gate == "none":
        # |silu''| <= 1/2: an error of v moves silu' by at most half of it
        dv, dvsize = dout * dsilu(v), np.abs(dout) * (expit(v) * (1 + np.abs(v)) + 0.5 * vsize)
    g, gsize = dv * w, dvsize * np.abs(w)

    def mean(a):
        m = a.reshape(T, groups, -1).mean(axis=2, keepdims=True)
        return np.broadcast_to(m, (T, groups, C // groups)).reshape(T, C)

    mg, mgh = (mean(g) if center else 0.0), mean(g * h)
    du = r * (g - mg - h * mgh)
    dusize = r * (gsize + (mean(gsize) if center else 0.0) + top * mean(gsize * top))
    if gate == "first":
        dx, sx = du * _silu(z), dusize * np.abs(_silu(z))
        dz, sz = du * x * dsilu(z), dusize * np.abs(x) * expit(z) * (1 + np.abs(z))
    elif gate == "last":
        dx, sx = du, dusize
        dz, sz = dout * v * dsilu(z), np.abs(dout) * vsize * expit(z) * (1 + np.abs(z))
    else:
        dx, sx, dz, sz = du, dusize, None, None
    return (dict(dx=dx, dz=dz, dweight=(dv * h).sum(axis=0), dbias=dv.sum(axis=0)),
            dict(dx=sx, dz=sz, dweight=(dvsize * top).sum(axis=0), dbias=dvsize.sum(axis=0)))
