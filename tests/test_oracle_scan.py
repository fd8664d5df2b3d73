"""The float64 oracle of the selective state space block's operators: closed forms, finite
differences, agreement with linear attention and with torch where it has the operator."""
import numpy as np
import pytest
import torch

from oracle import block as K
from oracle import scan as O

RNG = np.random.default_rng(0)


def normal(*shape):
    return RNG.standard_normal(shape)


def difference(f, x, i, e=1e-6):
    a, b = x.copy(), x.copy()
    a.flat[i] += e
    b.flat[i] -= e
    return (f(a) - f(b)) / (2 * e)


def check(f, x, grad, n=5):
    """Central differences of f at n places of x: off by rounding (1e-16 |f| / 1e-6) and by the third
    derivative (1e-12), so far below 1e-6 of the largest entry here."""
    at = RNG.choice(x.size, min(n, x.size), replace=False)
    for i in at:
        assert abs(difference(f, x, i) - grad.flat[i]) <= 1e-6 * max(1.0, np.abs(grad).max()), i


def test_rmsnorm_closed_forms():
    x, w, r = normal(3, 8), normal(8), normal(3, 8)
    y, h = O.rmsnorm(x, w, 1e-5, r)
    assert np.array_equal(h, x + r)
    assert np.allclose(y, torch.nn.functional.rms_norm(torch.tensor(x + r), (8,), torch.tensor(w), 1e-5).numpy(), atol=1e-13)
    c = np.full((1, 4), 3.0)
    assert np.allclose(O.rmsnorm(c, eps=0.0)[0], 1.0)
    assert np.array_equal(O.rmsnorm(np.zeros((2, 4)))[0], np.zeros((2, 4)))


def test_rmsnorm_gradients():
    x, w, dy, dh = normal(4, 6), normal(6), normal(4, 6), normal(4, 6)
    dx, dw = O.rmsnorm_backward(dy, x, w, 1e-3, dh)
    f = lambda x, w: (dy * O.rmsnorm(x, w, 1e-3)[0]).sum() + (dh * x).sum()  # noqa: E731
    check(lambda v: f(v, w), x, dx, 12)
    check(lambda v: f(x, v), w, dw)


def test_scales():
    y = np.array([[1.0, -4.0, 0.5, 2.0, 3.0], [0.0, 0.0, 0.0, 0.0, 0.0]])
    assert np.array_equal(O.scales(y, 2.0), [2.0, 2.0 ** -126])
    assert np.array_equal(O.scales(y, 2.0, 2)[0], [2.0, 1.0, 1.5])
    assert np.array_equal(O.spread(O.scales(y, 2.0, 2), 5, 2)[0], [2.0, 2.0, 1.0, 1.0, 1.5])
    assert O.spread(O.scales(y, 2.0), 5).shape == (2, 5)


@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_short_conv_against_torch_and_its_own_pieces(K):
    x, w, b = normal(11, 3), normal(3, K), normal(3)
    out, state = O.short_conv(x, w, b)
    t = torch.nn.functional.conv1d(torch.tensor(x.T[None]), torch.tensor(w[:, None]), torch.tensor(b), padding=K - 1, groups=3)
    assert np.allclose(out, t[0, :, :11].numpy().T, atol=1e-13)
    first, s = O.short_conv(x[:5], w, b, True)
    rest, s = O.short_conv(x[5:], w, b, True, s)
    whole, last = O.short_conv(x, w, b, True)
    assert np.allclose(np.concatenate((first, rest)), whole, atol=1e-13) and np.array_equal(s, last)
    assert np.array_equal(state, np.concatenate((np.zeros((K - 1, 3)), x))[11:])


@pytest.mark.parametrize("n", [1, 2, 9])
@pytest.mark.parametrize("silu", [False, True])
def test_short_conv_gradients(n, silu):
    K = 4
    x, w, b, s, dy, ds = normal(n, 3), normal(3, K), normal(3), normal(K - 1, 3), normal(n, 3), normal(K - 1, 3)
    got = O.short_conv_backward(dy, x, w, b, silu, s, ds)

    def f(x, w, b, s):
        out, last = O.short_conv(x, w, b, silu, s)
        return (dy * out).sum() + (ds * last).sum()
    check(lambda v: f(v, w, b, s), x, got[0])
    check(lambda v: f(x, v, b, s), w, got[1])
    check(lambda v: f(x, w, v, s), b, got[2])
    check(lambda v: f(x, w, b, v), s, got[3])


def scan_inputs(n, D=6, s=3, G=2):
    return dict(x=normal(n, D), dt=normal(n, D), A=-np.exp(normal(D, s)), B=normal(G, n, s), C=normal(G, n, s),
                skip=normal(D), bias=normal(D), z=normal(n, D), state=normal(D, s))


def test_selective_scan_is_linear_attention_where_decays_do_not_depend_on_the_state():
    """A the same for all states of a channel: each channel is a head with d_v = 1, q = C, k = B,
    v = D x and log decay D A."""
    n, D, s = 13, 4, 5
    p = scan_inputs(n, D, s, 1)
    p["A"] = np.repeat(p["A"][:, :1], s, 1)
    out, h = O.selective_scan(p["x"], p["dt"], p["A"], p["B"], p["C"], None, p["bias"], True, None, p["state"])
    step = np.logaddexp(p["dt"] + p["bias"], 0.0)
    o, S = K.linear_attention(np.repeat(p["C"], D, 0), np.repeat(p["B"], D, 0), (step * p["x"]).T[..., None],
                              (step * p["A"][:, 0]).T, 1.0, p["state"][..., None])
    assert np.allclose(out, o[..., 0].T, atol=1e-12) and np.allclose(h, S[..., 0], atol=1e-12)


def test_selective_scan_in_pieces_and_its_ends():
    p = scan_inputs(9)
    out, h = O.selective_scan(**p)
    cut = lambda a, b: {k: (v[:, a:b] if k in "BC" else v[a:b] if k in ("x", "dt", "z") else v) for k, v in p.items()}  # noqa: E731
    o1, s = O.selective_scan(**cut(0, 4))
    o2, s = O.selective_scan(**{**cut(4, 9), "state": s})
    assert np.allclose(np.concatenate((o1, o2)), out, atol=1e-12) and np.allclose(s, h, atol=1e-12)
    plain = O.selective_scan(**{**p, "z": None, "skip": None})[0]
    sg = 1.0 / (1.0 + np.exp(-p["z"]))
    assert np.allclose((plain + p["skip"] * p["x"]) * p["z"] * sg, out, atol=1e-12)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("n", [1, 7])
def test_selective_scan_gradients(n, softplus):
    p = scan_inputs(n)
    if not softplus:                  # steps as they are: positive, as the decays need them
        p["dt"], p["bias"] = np.abs(p["dt"]), np.abs(p["bias"])
    dy, ds = normal(n, 6), normal(6, 3)
    got = O.selective_scan_backward(dy, softplus=softplus, dstate=ds, **p)

    def f(**kw):
        out, h = O.selective_scan(softplus=softplus, **{**p, **kw})
        return (dy * out).sum() + (ds * h).sum()
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dD", bias="ddt_bias", z="dz", state="dstate_in")
    for k, g in names.items():
        check(lambda v: f(**{k: v}), p[k], got[g], 6)
