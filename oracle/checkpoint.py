"""fp64 oracle of the 8-bit activation checkpoints.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``. Blocks of 32
consecutive channels of a row share a step 2^s, the least power of two (s >=
-125) for which the block's largest magnitude rounds to at most 127 steps;
elements are whole numbers of steps, rounded to nearest, ties to even. A block
with an infinity or NaN reads as NaN.

Written with fp64 powers of two and a search over s, apart from the library's
arithmetic on exponent fields.
"""
from __future__ import annotations

import numpy as np

from oracle.conv import _f64

BLOCK = 32


def quantise(v):
    """(q, byte) of rows v (rows, channels): whole numbers and s + 127 per block."""
    v = _f64(v)
    rows, ch = v.shape
    nb = -(-ch // BLOCK)
    q = np.zeros((rows, ch))
    byte = np.zeros((rows, nb))
    for b in range(nb):
        blk = v[:, b * BLOCK:(b + 1) * BLOCK]
        with np.errstate(invalid="ignore", over="ignore"):
            top = np.abs(blk).max(axis=1)
            bad = ~np.isfinite(blk).all(axis=1)
            s = np.full(rows, -125)
            todo = ~bad
            while True:
                todo = todo & (np.rint(top * np.exp2(-s.astype(np.float64))) > 127)
                if not todo.any():
                    break
                s = s + todo
            part = np.rint(blk * np.exp2(-s.astype(np.float64))[:, None])
        q[:, b * BLOCK:(b + 1) * BLOCK] = np.where(bad[:, None], 0.0, part)
        byte[:, b] = np.where(bad, 255, s + 127)
    return q, byte


def values(q, byte):
    """The values a checkpoint stands for: 2^128, to which the top magnitudes
    of fp32 round, is infinity there."""
    q, byte = _f64(q), _f64(byte)
    step = np.repeat(np.where(byte == 255, np.nan, np.exp2(byte - 127)), BLOCK, axis=1)
    v = q * step[:, :q.shape[1]]
    return np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)


def kept(v):
    """What 8 bits keep of rows v."""
    return values(*quantise(v))
