"""The fp64 oracles of the operators around the SSD layer (group norm with
SiLU, the convolution front's backward pass, 8-bit checkpoints) against facts
fixed outside them: central differences of the forward definitions, torch's
own group norm, hand-worked blocks."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle.checkpoint import kept, quantise, values
from oracle.conv import conv_front
from oracle.conv_backward import conv_backward
from oracle.norm import norm, norm_backward


def _differences(f, v, h=1e-5):
    """Central differences of the scalar f at every element of v (in place)."""
    out = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = v[i]
        v[i] = old + h
        up = f()
        v[i] = old - h
        down = f()
        v[i] = old
        out[i] = (up - down) / (2 * h)
    return out


# A central difference is off by h^2/6 times a third derivative, of order one
# to ten here: 1e-10 .. 1e-9, and by rounding 1e-16 * |f| / h = 1e-10.
ATOL = 2e-8


@pytest.mark.parametrize("gate", ["first", "last", "none"])
@pytest.mark.parametrize("center", [False, True])
def test_norm_gradients_are_differences(gate, center):
    rng = np.random.default_rng(5)
    T, C, G, eps = 3, 12, 2, 1e-2
    x, d = rng.standard_normal((2, T, C))
    z = None if gate == "none" else rng.standard_normal((T, C))
    w, b = 1 + 0.3 * rng.standard_normal(C), 0.3 * rng.standard_normal(C)

    def loss():
        return float((norm(x, z, w, b, G, eps, center, gate)[0] * d).sum())

    g, _ = norm_backward(d, x, z, w, b, G, eps, center, gate)
    for name, v in (("dx", x), ("dz", z), ("dweight", w), ("dbias", b)):
        if v is not None:
            assert np.allclose(g[name], _differences(loss, v), rtol=0, atol=ATOL), name
    assert (g["dz"] is None) == (gate == "none")


@pytest.mark.parametrize("groups", [1, 3])
def test_centred_norm_is_torch_group_norm(groups):
    rng = np.random.default_rng(6)
    x, w, b = rng.standard_normal((7, 24)), rng.standard_normal(24), rng.standard_normal(24)
    t = torch.nn.functional.group_norm(torch.from_numpy(x), groups, torch.from_numpy(w),
                                       torch.from_numpy(b), 1e-5)
    want = torch.nn.functional.silu(t).numpy()
    got, _ = norm(x, None, w, b, groups, 1e-5, True, "none")
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_norm_of_a_constant_row():
    """u = c: without centring h = c / sqrt(c^2 + eps); with it 0."""
    x = np.full((1, 8), 3.0)
    got, _ = norm(x, None, None, None, 1, 0.25, False, "none")
    h = 3.0 / np.sqrt(9.25)
    assert np.allclose(got, h / (1 + np.exp(-h)), rtol=1e-14)
    got, _ = norm(x, np.ones((1, 8)), None, None, 1, 0.25, True, "last")
    assert np.array_equal(got, np.zeros((1, 8)))


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("bounds", [[(0, 5), (5, 5), (5, 6), (6, 8)], [(0, 4), (4, 8)]])
def test_conv_gradients_are_differences(K, bounds):
    rng = np.random.default_rng(7 + K)
    T, ch, S = 8, 4, len(bounds)
    u, d = rng.standard_normal((2, T, ch))
    w, b = rng.standard_normal((ch, K)), rng.standard_normal(ch)
    h, dh = rng.standard_normal((2, S, K - 1, ch))

    def loss():
        x, B, C, ho = conv_front(u, w, b, bounds, ch, 0, h)
        return float((x * d).sum() + (ho * dh).sum())

    g, _ = conv_backward(u, w, b, bounds, d, h, dh)
    for name, v in (("dxbc", u), ("dweight", w), ("dbias", b), ("dhistory", h)):
        assert np.allclose(g[name], _differences(loss, v), rtol=0, atol=ATOL), name


def test_checkpoint_worked_blocks():
    """Blocks worked by hand: 127 fits step 1 exactly; 127.5 rounds to 128 and
    takes step 2; 1.0 takes step 1/64 (64 steps; with 1/128 it would be 128);
    zeros take the least step; an infinity spoils its block only."""
    v = np.zeros((5, 40))
    v[0, 3], v[0, 4], v[0, 5] = 127.0, 0.5, 1.5     # ties go to even: 0, 2
    v[1, 0], v[1, 1] = 127.5, 1.0                    # step 2: 63.75 -> 64; 0.5 -> 0
    v[2, 0], v[2, 35] = -1.0, 3.0
    v[4, 2], v[4, 33] = np.inf, 1.0
    q, byte = quantise(v)
    assert byte[0, 0] == 127 and list(q[0, 3:6]) == [127, 0, 2]
    assert byte[1, 0] == 128 and list(q[1, :2]) == [64, 0]
    assert byte[2, 0] == 127 - 6 and q[2, 0] == -64
    assert byte[2, 1] == 127 - 5 and q[2, 35] == 96
    assert byte[3, 0] == 2 and not q[3].any()
    assert byte[4, 0] == 255 and not q[4, :32].any() and byte[4, 1] == 127 - 6
    back = values(q, byte)
    assert np.isnan(back[4, :32]).all() and back[4, 33] == 1.0


def test_checkpoint_is_within_half_a_step_and_minimal():
    rng = np.random.default_rng(9)
    v = rng.standard_normal((50, 96)) * np.exp(4 * rng.standard_normal((50, 96)))
    q, byte = quantise(v)
    step = np.repeat(np.exp2(byte - 127), 32, axis=1)
    assert np.abs(q).max() <= 127 and (np.abs(kept(v) - v) <= step / 2).all()
    # half the step would need more than 127
    top = np.abs(v).reshape(50, 3, 32).max(axis=2)
    assert (np.rint(2 * top / np.exp2(byte - 127)) > 127).all()


def test_checkpoint_at_the_ends_of_fp32():
    big = float(np.finfo(np.float32).max)
    q, byte = quantise(np.array([[big] * 32, [1e-45] * 32, [2.0 ** -119] * 32]))
    assert list(byte[:, 0]) == [249, 2, 127 - 125]
    assert q[0, 0] == 64 and q[1, 0] == 0 and q[2, 0] == 64
    # 64 steps of 2^122 are past fp32's range, as that magnitude rounded to 7 bits is
    assert values(q, byte)[0, 0] == np.inf and values(-q, byte)[0, 0] == -np.inf
