"""The operators of a selective state space block, in float64 numpy: root-mean-square norm (with
outputs in 8 bits), the short causal convolution and the selective scan, each with its gradients. One
sequence at a time where there are tokens."""
from __future__ import annotations

import numpy as np

from .retention import to64


def rmsnorm(x, weight=None, eps=1e-5, residual=None):
    """(y, sum) of rows x [..., d] (+ residual)."""
    h = to64(x) + (0.0 if residual is None else to64(residual))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * to64(weight)), h


def rmsnorm_backward(dout, x, weight=None, eps=1e-5, dsum=None):
    """(dx, dweight) of sum(dout * rmsnorm(x)) + sum(dsum * x)."""
    x, dy = to64(x), to64(dout)
    d = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dy if weight is None else dy * to64(weight)
    dx = g * r - x * r ** 3 * (g * x).sum(-1, keepdims=True) / d
    if dsum is not None:
        dx = dx + to64(dsum)
    return dx, (dy * x * r).sum(tuple(range(x.ndim - 1)))


def scales(y, most, group=0):
    """The scale of each row of y [..., d], or of each ``group`` columns of it."""
    y = np.abs(to64(y))
    if not group:
        return np.maximum(y.max(-1) / most, 2.0 ** -126)
    parts = [y[..., i:i + group].max(-1) for i in range(0, y.shape[-1], group)]
    return np.maximum(np.stack(parts, -1) / most, 2.0 ** -126)


def spread(scale, d, group=0):
    """The scale of each of d columns."""
    return np.repeat(scale, group, -1)[..., :d] if group else np.repeat(scale[..., None], d, -1)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def short_conv(x, weight, bias=None, silu=False, state=None):
    """(out, state) of x [n, D], weight [D, K], state [K - 1, D] or None."""
    x, w = to64(x), to64(weight)
    n, K = len(x), w.shape[1]
    rows = np.concatenate((np.zeros((K - 1, x.shape[1])) if state is None else to64(state), x))
    u = np.zeros_like(x) + (0.0 if bias is None else to64(bias))
    for t in range(n):
        u[t] += (rows[t:t + K] * w.T).sum(0)
    return (u * sigmoid(u) if silu else u), rows[n:]


def short_conv_backward(dout, x, weight, bias=None, silu=False, state=None, dstate=None):
    """(dx, dweight, dbias, gradient of the first state)."""
    x, w, du = to64(x), to64(weight), to64(dout).copy()
    n, K = len(x), w.shape[1]
    rows = np.concatenate((np.zeros((K - 1, x.shape[1])) if state is None else to64(state), x))
    if silu:
        u, _ = short_conv(x, weight, bias, False, state)
        s = sigmoid(u)
        du *= s + u * s * (1.0 - s)
    drows, dw = np.zeros_like(rows), np.zeros_like(w)
    for t in range(n):
        drows[t:t + K] += w.T * du[t]
        dw += (rows[t:t + K] * du[t]).T
    if dstate is not None:
        drows[n:] += to64(dstate)
    return drows[K - 1:], dw, du.sum(0), drows[:K - 1]


def _step(dt, bias, softplus):
    v = to64(dt) + (0.0 if bias is None else to64(bias))
    return (np.logaddexp(v, 0.0) if softplus else v), v


def _channels(B, D):
    """[G, n, states] -> [n, D, states]."""
    return np.repeat(to64(B), D // len(B), 0).transpose(1, 0, 2)


def selective_scan(x, dt, A, B, C, skip=None, bias=None, softplus=True, z=None, state=None, keep=None):
    """(out, state) of one sequence: x, dt, z [n, D], A [D, s], B, C [G, n, s], state [D, s] or None.
    ``keep``, a list, receives the state after each token."""
    x, A = to64(x), to64(A)
    n, D = x.shape
    B, C = _channels(B, D), _channels(C, D)
    step, _ = _step(dt, bias, softplus)
    h = np.zeros_like(A) if state is None else to64(state).copy()
    y = np.zeros_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(n):
            h = np.exp(step[t][:, None] * A) * h + (step[t] * x[t])[:, None] * B[t]
            y[t] = (C[t] * h).sum(1)
            if keep is not None:
                keep.append(h)
        if skip is not None:
            y = y + to64(skip) * x
        return (y if z is None else y * to64(z) * sigmoid(to64(z))), h


def selective_scan_backward(dout, x, dt, A, B, C, skip=None, bias=None, softplus=True, z=None, state=None, dstate=None):
    """A dict of the gradients of sum(dout * out) + sum(dstate * final state) of one sequence."""
    x, A, dy = to64(x), to64(A), to64(dout)
    n, D = x.shape
    G = len(B)
    first = np.zeros_like(A) if state is None else to64(state)
    kept = []
    y, _ = selective_scan(x, dt, A, B, C, skip, bias, softplus, None, first, kept)
    B, C = _channels(B, D), _channels(C, D)
    step, v = _step(dt, bias, softplus)
    got = {}
    if z is not None:
        zz = to64(z)
        s = sigmoid(zz)
        got["dz"] = dy * y * (s + zz * s * (1.0 - s))
        dy = dy * zz * s
    g = np.zeros_like(A) if dstate is None else to64(dstate).copy()
    dx, dstep, dA = np.zeros_like(x), np.zeros_like(x), np.zeros_like(A)
    dB, dC = (np.zeros((G, n, A.shape[1])) for _ in range(2))
    for t in reversed(range(n)):
        g = g + C[t] * dy[t][:, None]
        a = np.exp(step[t][:, None] * A)
        before = kept[t - 1] if t else first
        da = g * before * a
        dC[:, t] = (kept[t] * dy[t][:, None]).reshape(G, -1, A.shape[1]).sum(1)
        dB[:, t] = (g * (step[t] * x[t])[:, None]).reshape(G, -1, A.shape[1]).sum(1)
        du = (g * B[t]).sum(1)
        dx[t] = du * step[t]
        dstep[t] = du * x[t] + (da * A).sum(1)
        dA += da * step[t][:, None]
        g = g * a
    if skip is not None:
        dx += to64(skip) * dy
        got["dD"] = (dy * x).sum(0)
    ddt = dstep * sigmoid(v) if softplus else dstep
    got.update(dx=dx, ddt=ddt, ddt_bias=ddt.sum(0), dA=dA, dB=dB, dC=dC, dstate_in=g)
    return got
