"""Pins of the float64 oracle of the operators around retention (CPU)."""
import numpy as np
import pytest

import oracle as O
from oracle import block as K


def test_layernorm_rows_have_mean_bias_and_unit_variance():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 5, 33)) * 4 + 7
    y, h = K.layernorm(x, eps=0.0)
    assert np.array_equal(h, x)
    assert np.abs(y.mean(-1)).max() < 1e-13 and np.abs((y * y).mean(-1) - 1).max() < 1e-13
    y, h = K.layernorm(x, np.full(33, 2.0), np.full(33, -1.0), 0.0, residual=-x)
    assert np.isnan(y).all() and not h.any()          # 0 / 0: eps = 0 on a constant row
    y, _ = K.layernorm(x, np.full(33, 2.0), np.full(33, -1.0), 1e-5, residual=-x)
    assert np.array_equal(y, np.full_like(x, -1.0))


@pytest.mark.parametrize("affine", [False, True])
def test_layernorm_gradients_against_differences(affine):
    rng = np.random.default_rng(1)
    x, dy, dh = (rng.standard_normal((4, 7)) for _ in range(3))
    w = rng.standard_normal(7) if affine else None
    b = rng.standard_normal(7) if affine else None

    def loss(x_, w_, b_):
        y, h = K.layernorm(x_, w_, b_, 1e-3)
        return (y * dy).sum() + (h * dh).sum()

    dx, dw, db = K.layernorm_backward(dy, x, w, 1e-3, dh)
    e = 1e-6

    def num(a, f):
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += e
            dn[i] -= e
            g[i] = (f(up) - f(dn)) / (2 * e)
        return g

    assert np.abs(num(x, lambda a: loss(a, w, b)) - dx).max() < 1e-7
    if affine:
        assert np.abs(num(w, lambda a: loss(x, a, b)) - dw).max() < 1e-7
        assert np.abs(num(b, lambda a: loss(x, w, a)) - db).max() < 1e-7


@pytest.mark.parametrize("half", [False, True])
def test_rotary_closed_forms(half):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 3, 5, 10))
    theta = np.array([1.0, 0.3, 0.01])
    pos = rng.integers(0, 1000, (2, 5))
    y = K.rotary(x, theta, pos, half)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    pair = (lambda a, j: (a[..., j], a[..., j + 3])) if half else (lambda a, j: (a[..., 2 * j], a[..., 2 * j + 1]))
    for j in range(3):
        (a, b), (c, d) = pair(x, j), pair(y, j)
        ang = (pos * theta[j])[:, None]
        assert np.abs(c - (a * np.cos(ang) - b * np.sin(ang))).max() < 1e-12
        assert np.abs(d - (a * np.sin(ang) + b * np.cos(ang))).max() < 1e-12
    assert np.abs(K.rotary(y, theta, pos, half, inverse=True) - x).max() < 1e-12
    # the transpose: <dy, R x> = <R^T dy, x>, magnitude included
    dy = rng.standard_normal(x.shape)
    lhs = (dy * K.rotary(x, theta, pos, half, magnitude=1.3)).sum()
    rhs = (K.rotary(dy, theta, pos, half, inverse=True, magnitude=1.3) * x).sum()
    # (coordinates that are not turned are not scaled either)
    assert abs(lhs - rhs) < 1e-10


def test_rotary_agrees_with_retentions_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 2, 6, 8))
    theta = np.array([1.0, 0.5, 0.2, 0.1])
    want = O.rotate(x, np.arange(6) + 41, theta)
    assert np.abs(K.rotary(x, theta, np.arange(6)[None] + 41) - want).max() < 1e-12


def test_linear_attention_with_constant_decay_is_retention():
    rng = np.random.default_rng(4)
    q, k = rng.standard_normal((2, 1, 3, 20, 4))
    v = rng.standard_normal((1, 3, 20, 5))
    S0 = rng.standard_normal((1, 3, 4, 5))
    gamma = np.array([1.0, 0.9, 0.3])
    want, S = O.recurrent(q, k, v, gamma, np.zeros(2), 0, 0.7, S0)
    got, S1 = K.linear_attention(q[0], k[0], v[0], np.log(gamma)[:, None].repeat(20, 1), 0.7, S0[0])
    assert np.abs(got - want[0]).max() < 1e-12 and np.abs(S1 - S[0]).max() < 1e-12


def test_linear_attention_reset_and_shared_heads():
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((2, 1, 9, 3))
    v = rng.standard_normal((4, 9, 2))
    g = -rng.random((4, 9))
    g[:, 5] = -np.inf                                  # clears the state before token 5
    o, S = K.linear_attention(q, k, v, g)
    o2, S2 = K.linear_attention(q[:, 5:], k[:, 5:], v[:, 5:], g[:, 5:])
    assert np.array_equal(o[:, 5:], o2) and np.array_equal(S, S2)
    for h in range(4):                                 # direct sum over earlier tokens
        for t in range(5):
            want = sum(np.exp(g[h, s + 1:t + 1].sum()) * (q[0, t] @ k[0, s]) * v[h, s] for s in range(t + 1))
            assert np.abs(o[h, t] - want).max() < 1e-12
