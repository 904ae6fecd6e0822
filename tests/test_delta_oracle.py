"""The fp64 oracles of the gated delta rule and of the norm and rotation of keys
and queries, against facts fixed outside them: central differences of the forward
definitions, the layer's own recurrence, hand-worked cases."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from oracle.delta import bc_norm, bc_norm_backward, delta_backward, delta_rule
from test_layer_oracle import ATOL, _differences


def _problem(rng, T, H, P, N, G, S):
    unit = lambda v: v / np.linalg.norm(v, axis=-1, keepdims=True)
    return dict(x=rng.standard_normal((T, H, P)), g=-rng.uniform(0, 1, (T, H)),
                beta=rng.uniform(0, 1.5, (T, H)), B=unit(rng.standard_normal((T, G, N))),
                C=rng.standard_normal((T, G, N)), h0=rng.standard_normal((S, H, P, N)))


def test_orthonormal_keys_only_add():
    """With orthonormal keys and no initial state nothing is stored for a key before
    it comes: the layer's recurrence with values beta x and a step of one."""
    rng = np.random.default_rng(1)
    T, H, P, N = 8, 3, 4, 8
    p = _problem(rng, T, H, P, N, 1, 1)
    p["B"] = np.linalg.qr(rng.standard_normal((N, N)))[0][:, None, :]
    p["g"][:] = p["g"][:1]
    y, h = delta_rule(p["x"], p["g"], p["beta"], p["B"], p["C"])
    want, hw = oracle.ssd_recurrence(p["x"] * p["beta"][..., None], np.ones((T, H)), p["g"][0],
                                     p["B"], p["C"])
    assert np.allclose(y, want, rtol=0, atol=1e-13) and np.allclose(h, hw, rtol=0, atol=1e-13)


def test_a_key_written_again_is_replaced():
    k = np.array([[[0.6, 0.8]]])
    x = np.array([[[1.0]], [[5.0]]])
    y, h = delta_rule(x, np.zeros((2, 1)), np.ones((2, 1)), np.repeat(k, 2, 0), np.repeat(k, 2, 0))
    assert np.allclose(y[:, 0, 0], [1, 5]) and np.allclose(h[0, 0], 5 * k[0])


def test_nothing_written_without_beta_and_minus_infinity_resets():
    rng = np.random.default_rng(2)
    p = _problem(rng, 3, 2, 3, 4, 2, 1)
    y, h = delta_rule(p["x"], p["g"], 0 * p["beta"], p["B"], p["C"], p["h0"])
    assert np.allclose(h[0], p["h0"][0] * np.exp(p["g"].sum(0))[:, None, None])
    p["g"][2] = -np.inf
    last = lambda v: v[2:]
    y, h = delta_rule(p["x"], p["g"], p["beta"], p["B"], p["C"], p["h0"])
    y2, h2 = delta_rule(*(last(p[k]) for k in ("x", "g", "beta", "B", "C")))
    assert np.allclose(y[2:], y2) and np.allclose(h, h2)


def test_gradients_are_differences():
    rng = np.random.default_rng(3)
    lens, H, P, N, G = [3, 0, 2], 4, 2, 3, 2
    p = _problem(rng, 5, H, P, N, G, 3)
    dy, dhT = rng.standard_normal((5, H, P)), rng.standard_normal((3, H, P, N))

    def loss():
        y, h = delta_rule(p["x"], p["g"], p["beta"], p["B"], p["C"], p["h0"], lens)
        return float((y * dy).sum() + (h * dhT).sum())

    d = delta_backward(p["x"], p["g"], p["beta"], p["B"], p["C"], p["h0"], lens, dy, dhT)
    for name, k in (("dx", "x"), ("dg", "g"), ("dbeta", "beta"), ("dB", "B"), ("dC", "C"),
                    ("dinitial_state", "h0")):
        assert np.allclose(d[name], _differences(loss, p[k]), rtol=0, atol=ATOL), name


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients_are_differences(unit, interleaved):
    rng = np.random.default_rng(4)
    x, d = rng.standard_normal((2, 4, 2, 12))
    w, freqs = rng.standard_normal(12), np.array([0.3, 0.01, 1.0, 2.0])
    kw = dict(positions=np.array([5, 9]), freqs=freqs, eps=0.1, unit=unit, interleaved=interleaved)
    loss = lambda: float((bc_norm(x, w, **kw)[0] * d).sum())
    (dx, dw), _ = bc_norm_backward(d, x, w, **kw)
    assert np.allclose(dx, _differences(loss, x), rtol=0, atol=ATOL)
    assert np.allclose(dw, _differences(loss, w), rtol=0, atol=ATOL)


def test_norm_is_a_rotation_by_the_distance():
    """Lengths stay, and the product of a turned key and query depends on the
    difference of their positions only."""
    rng = np.random.default_rng(5)
    x = np.repeat(rng.standard_normal((1, 2, 8)), 4, axis=0)
    freqs = np.array([1.0, 0.1, 0.01])
    out, _ = bc_norm(x, None, np.array([0, 3, 100, 103]), freqs, eps=0.0, unit=True)
    assert np.allclose(np.linalg.norm(out, axis=2), 1)
    assert np.allclose(out[0, 0] @ out[1, 1], out[2, 0] @ out[3, 1])
    assert not np.allclose(out[0, 0] @ out[1, 1], out[0, 0] @ out[2, 1])
    assert np.allclose(out[0], x[0] / np.linalg.norm(x[0], axis=1, keepdims=True))
    flat, _ = bc_norm(x, None, eps=0.0)
    assert np.allclose((flat ** 2).mean(axis=2), 1)
    inter, _ = bc_norm(x, None, np.array([0, 3, 100, 103]), freqs, eps=0.0, unit=True,
                       interleaved=True)
    order = [0, 2, 4, 1, 3, 5, 6, 7]      # channels of pairs (2i, 2i + 1) as (i, i + 3)
    want, _ = bc_norm(x[..., order], None, np.array([0, 3, 100, 103]), freqs, eps=0.0, unit=True)
    assert np.allclose(inter[..., order], want)
