"""The operators around retention, in float64 numpy: layer norm and its gradients, rotary
positions, linear attention with a decay per head and token."""
from __future__ import annotations

import numpy as np

from .retention import to64


def layernorm(x, weight=None, bias=None, eps=1e-5, residual=None):
    """(out, sum) of rows x [..., d] (+ residual): biased variance, eps inside the root."""
    h = to64(x) + (0.0 if residual is None else to64(residual))
    c = h - h.mean(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        y = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * to64(weight)
    if bias is not None:
        y = y + to64(bias)
    return y, h


def layernorm_backward(dout, x, weight=None, eps=1e-5, dsum=None):
    """(dx, dweight, dbias) of sum(dout * layernorm(x)) + sum(dsum * x)."""
    x, dy = to64(x), to64(dout)
    d = x.shape[-1]
    c = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    g = dy if weight is None else dy * to64(weight)
    # through y = c r(c), then through c = x - mean(x)
    dc = g * r - c * r ** 3 * (g * c).sum(-1, keepdims=True) / d
    dx = dc - dc.mean(-1, keepdims=True)
    if dsum is not None:
        dx = dx + to64(dsum)
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * c * r).sum(rows), dy.sum(rows)


def rotary(x, theta, pos, half=False, inverse=False, magnitude=1.0):
    """x [B, H, N, d] with token positions pos [B, N]: pair j of the first 2 len(theta)
    coordinates times magnitude * exp(+- i p theta_j)."""
    y = to64(x).copy()
    n = len(theta)
    a = np.asarray(pos, dtype=np.float64)[:, None, :, None] * np.asarray(theta, dtype=np.float64)
    z = magnitude * np.exp((-1j if inverse else 1j) * a)
    i, j = (slice(0, n), slice(n, 2 * n)) if half else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    w = (y[..., i] + 1j * y[..., j]) * z
    y[..., i], y[..., j] = w.real, w.imag
    return y


def linear_attention(q, k, v, log_decay, scale=1.0, state=None):
    """One sequence, token by token: q [H_q, n, d_k], k [H_k, n, d_k], v [H_v, n, d_v],
    log_decay [H, n], state [H, d_k, d_v] or None. Returns (out [H, n, d_v], final state)."""
    g = to64(log_decay)
    H, n = g.shape
    q, k, v = (np.repeat(to64(x), H // len(x), 0) for x in (q, k, v))
    S = np.zeros((H, q.shape[-1], v.shape[-1])) if state is None else to64(state).copy()
    out = np.zeros((H, n, v.shape[-1]))
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(n):
            S = np.exp(g[:, t])[:, None, None] * S + k[:, t, :, None] * v[:, t, None, :]
            out[:, t] = scale * (q[:, t, :, None] * S).sum(1)
    return out, S
