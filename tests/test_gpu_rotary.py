"""Rotary positions on the GPU against the float64 oracle.

Tolerance: the reduced angle in float32 is off by at most 2^-23 (half a step below 4), the
float32 sine and cosine by 2 u, the magnitude and the two products and their sum by 4 u:
below 8 u magnitude (|a| + |b|) for the pair (a, b), u = 2^-24; half a step of the type added."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import block as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def heads(gen, B, H, N, d, dt, token_major):
    shape = (B, N, H, d) if token_major else (B, H, N, d)
    x = torch.randn(shape, generator=gen).to(dt).to(DEV)
    return x.transpose(1, 2) if token_major else x


def partner(x, n, half):
    a = np.abs(np64(x)).copy()
    i, j = (slice(0, n), slice(n, 2 * n)) if half else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    s = a[..., i] + a[..., j]
    a[...] = 0
    a[..., i], a[..., j] = s, s
    return a


def check(got, x, theta, pos, half, inverse, m):
    want = K.rotary(x, theta, pos, half, inverse, m)
    off = np.abs(np64(got) - want)
    h = torch.finfo(x.dtype).eps / 2
    tol = 8 * U * m * partner(x, len(theta), half) + 1.01 * h * np.abs(want) * (np.arange(x.shape[-1]) < 2 * len(theta))
    assert (off <= tol).all(), (off - tol).max()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot", [
    (1, 1, 1, 0, 2, 2), (3, 1, 8, 2, 128, 128), (2, 33, 3, 1, 64, 32), (1, 70, 5, 5, 80, 6), (2, 19, 4, 4, 96, 48),
    (1, 130, 2, 2, 256, 256), (64, 1, 32, 8, 128, 64), (2, 257, 1, 1, 33, 30), (1, 9, 2, 1, 512, 256), (1, 2100, 4, 1, 128, 128),
    (2, 40, 3, 2, 24, 24), (1, 17, 40, 1, 40, 16)])
def test_against_the_oracle(kind, half, B, N, Hq, Hk, d, rot):
    g = torch.Generator().manual_seed(B * 100 + N + rot)
    rng = np.random.default_rng(N + rot)
    theta = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    for tm, inverse, m in ((False, False, 1.0), (True, False, 1.25), (True, True, 0.5), (False, True, 1.0)):
        q = heads(g, B, Hq, N, d, DT[kind], tm)
        k = heads(g, B, Hk, N, d, DT[kind], not tm) if Hk else None
        first = rng.integers(0, 1 << 20, B)
        each = rng.integers(0, 1 << 20, (B, N))
        for pos, kw in ((np.arange(N)[None] + np.full((B, 1), 65000), dict(pos0=65000)),
                        (first[:, None] + np.arange(N), dict(pos=torch.tensor(first, device=DEV))),
                        (each, dict(pos=torch.tensor(each, device=DEV)))):
            got = rn().rn_rotary(q, k, theta, half=half, inverse=inverse, magnitude=m, **kw)
            qo, ko = got if Hk else (got, None)
            check(qo, q, theta, pos, half, inverse, m)
            assert qo.shape == q.shape and qo.dtype == q.dtype
            if Hk:
                check(ko, k, theta, pos, half, inverse, m)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("kind,off", [("bf16", 0), ("bf16", 1), ("f32", 1)])
def test_views_of_a_projection_in_place(half, kind, off):
    """q and k as slices of one buffer [B, N, (Hq + Hk + Hv) d + off], rotated in place: the rest
    of the buffer keeps its bits."""
    B, N, Hq, Hk, d, rot = 2, 50, 4, 2, 64, 32
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(B, N, (Hq + 2 * Hk) * d + off, generator=g).to(DT[kind]).to(DEV)
    before = buf.clone()
    cut = lambda b, h0, h: b[..., off + h0 * d:off + (h0 + h) * d].unflatten(-1, (h, d)).transpose(1, 2)  # noqa: E731
    q, k = cut(buf, 0, Hq), cut(buf, Hq, Hk)
    theta = 100.0 ** (-2.0 * np.arange(rot // 2) / rot)
    want_q, want_k = rn().rn_rotary(q, k, theta, pos0=7, half=half)
    a, b = rn().rn_rotary(q, k, theta, pos0=7, half=half, q_out=q, k_out=k)
    assert a is q and b is k and torch.equal(q, want_q) and torch.equal(k, want_k)
    check(q, cut(before, 0, Hq), theta, np.arange(N)[None].repeat(B, 0) + 7, half, False, 1.0)
    assert torch.equal(buf[..., off + (Hq + Hk) * d:], before[..., off + (Hq + Hk) * d:])
    assert torch.equal(q[..., rot:], cut(before, 0, Hq)[..., rot:])
    # every token the same input: a stride of 0
    one = q[:, :, :1]
    same = rn().rn_rotary(one.expand(B, Hq, N, d), None, theta, pos0=7, half=half)
    assert torch.equal(same, rn().rn_rotary(one.expand(B, Hq, N, d).contiguous(), None, theta, pos0=7, half=half))


def test_there_and_back_and_gradient():
    """R^T R = magnitude^2 on turned pairs; and <dy, R x> = <R^T dy, x>."""
    g = torch.Generator().manual_seed(4)
    x, dy = (torch.randn(2, 3, 40, 64, generator=g).to(DEV) for _ in range(2))
    theta, m = rn().rn_rotary_frequencies(48, kind="by_parts", factor=4.0, length=512)
    for half in (False, True):
        kw = dict(half=half, magnitude=m, pos0=99)
        y = rn().rn_rotary(x, None, theta, **kw)
        back = rn().rn_rotary(y, None, theta, inverse=True, **kw)
        scale = torch.ones(64, device=DEV)
        scale[:48] = m * m
        assert ((back - x * scale).abs() <= 64 * U * m * m * x.abs().max()).all()
        dx = rn().rn_rotary(dy, None, theta, inverse=True, **kw)
        lhs, rhs = (dy.double() * y).sum().item(), (dx.double() * x).sum().item()
        assert abs(lhs - rhs) <= 16 * U * m * (dy.double().abs() * x.double().abs().amax()).sum().item()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_rotated_tensors_feed_retention(kind):
    """Retention with theta = 0 on tensors turned here equals retention with its own rotation:
    exactly the same products in float32 up to the rotation's roundings; for bf16 the turned
    values are rounded once more (half a step of each of q and k)."""
    w = W.Workload("t", "chunkwise", B=2, H=2, N=100, d_k=32, d_v=32, dtype=kind, chunk=32, qkv_std=0.25, seed=9)
    x = W.make_inputs(w)
    q, k, v = (x[n].to(DEV) for n in "qkv")
    own, _ = rn().rn_retention_chunkwise(q, k, v, x["gamma"], x["theta"], 32, pos0=500, out_dtype=torch.float32)
    tq, tk = rn().rn_rotary(q, k, x["theta"].astype(np.float64), pos0=500)
    got, _ = rn().rn_retention_chunkwise(tq, tk, v, x["gamma"], np.zeros(16), 32, out_dtype=torch.float32)
    # |score| terms: sum over pairs of |q||k|, weighted by |v| and the decays' sum
    mass, _ = rn().rn_retention_chunkwise(q.abs(), k.abs(), v.abs(), x["gamma"], np.zeros(16), 32, out_dtype=torch.float32)
    h = torch.finfo(DT[kind]).eps / 2 if kind == "bf16" else 64 * U
    assert ((got - own).abs() <= 2 * 2.1 * h * mass * 2).all()      # a turned pair: up to sqrt 2 of |a| + |b| each


@pytest.mark.parametrize("half", [False, True])
def test_far_positions_and_many_tokens(half):
    """Positions beyond 2^32 (the product with theta is the same float64 number on both sides),
    and more tokens than one round of blocks."""
    g = torch.Generator().manual_seed(6)
    theta = np.array([1.0, 0.37, 1e-3, 1e-9])
    x = torch.randn(2, 1, 5, 8, generator=g).to(DEV)
    far = torch.tensor([(1 << 33) + 1, (1 << 36) - 7], device=DEV)
    check(rn().rn_rotary(x, None, theta, pos=far, half=half), x, theta, far.cpu().numpy()[:, None] + np.arange(5), half, False, 1.0)
    x = torch.randn(3, 1, 30001, 8, generator=g).to(DEV)
    check(rn().rn_rotary(x, None, theta, pos0=5, half=half), x, theta, np.arange(30001)[None].repeat(3, 0) + 5, half, False, 1.0)


def test_refusals():
    q = torch.zeros(2, 4, 8, 64, device=DEV)
    th = np.ones(32)
    for kw in (dict(k=torch.zeros(2, 4, 9, 64, device=DEV)), dict(k=q.bfloat16()), dict(pos=torch.zeros(3, dtype=torch.int64, device=DEV)),
               dict(pos=torch.zeros(2, dtype=torch.int32, device=DEV)), dict(pos=torch.zeros(2, dtype=torch.int64)),
               dict(q_out=torch.zeros(2, 4, 8, 65, device=DEV)), dict(k_out=q), dict(theta=None), dict(theta=np.ones((2, 2)))):
        with pytest.raises(ValueError):
            rn().rn_rotary(q, **{"theta": th, **kw})
    with pytest.raises(ValueError):
        rn().rn_rotary(q.transpose(2, 3), None, th)
    with pytest.raises(rn().RnError):
        rn().rn_rotary(q, None, np.ones(33))
    with pytest.raises(rn().RnError):
        rn().rn_rotary(q, None, th, q_out=torch.zeros(1, 4, 8, 64, device=DEV).expand(2, 4, 8, 64))
    with pytest.raises(TypeError):
        rn().rn_rotary(q.half(), None, th)
    with pytest.raises(ValueError):
        rn().rn_rotary(q[:, :, :0], None, th)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("d,rot", [(102, 102), (102, 4), (66, 50), (36, 12), (44, 24), (40, 40)])
def test_pieces_of_every_size_at_any_address(kind, half, d, rot):
    """Head sizes that pieces of 2, 4 and 8 elements divide, in views that start one element in
    and whose rows are an odd number of elements apart: nothing around them is written."""
    B, N, H = 2, 21, 3
    g = torch.Generator().manual_seed(d + rot)
    theta = 50.0 ** (-2.0 * np.arange(rot // 2) / rot)
    wide = torch.randn(B, N, H, d + 3, generator=g).to(DT[kind]).to(DEV)
    x = wide[..., 1:1 + d].transpose(1, 2)
    into = torch.full((B, H, N, d + 1), 7.0, dtype=DT[kind], device=DEV)
    got = rn().rn_rotary(x, None, theta, pos0=3, half=half, q_out=into[..., 1:])
    check(got, x, theta, np.arange(N)[None].repeat(B, 0) + 3, half, False, 1.0)
    assert torch.equal(got[..., rot:], x[..., rot:]) and (into[..., 0] == 7.0).all()
    before = wide.clone()
    rn().rn_rotary(x, None, theta, pos0=3, half=half, q_out=x)
    assert torch.equal(x, got)
    assert torch.equal(wide[..., 0], before[..., 0]) and torch.equal(wide[..., 1 + d:], before[..., 1 + d:])


@pytest.mark.parametrize("half", [False, True])
def test_float32_keeps_what_the_angles_have(half):
    """The error in the mean square. One rounding is off by at most U / sqrt(3) of its value there. A
    turned value a c - b s takes one of the sum, one of one of its two products (half of the square),
    and those of c and s (each half of it): sqrt(2.5) U / sqrt(3) together. An angle rounded to
    float32 would add about 0.77 U (angles spread over a turn), 1.2 U with these."""
    B, H, N, d = 2, 4, 3000, 64
    g = torch.Generator().manual_seed(31)
    x = torch.randn(B, H, N, d, generator=g).to(DEV)
    theta = 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    got = rn().rn_rotary(x, None, theta, pos0=12345, half=half)
    want = K.rotary(x.cpu(), theta, np.arange(N)[None].repeat(B, 0) + 12345, half)
    off = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert off <= (2.5 / 3) ** 0.5 * U, off / U


def test_more_tiles_than_one_grid_axis_takes():
    """2^29 + 37 tokens (2 GiB): tokens from all over the call equal those of short calls at their
    positions, bit by bit."""
    N = (1 << 29) + 37
    one = torch.randn(1, 1, 1, 2, generator=torch.Generator().manual_seed(32)).bfloat16().to(DEV)
    theta = np.array([0.37])
    out = torch.empty(1, 1, N, 2, dtype=torch.bfloat16, device=DEV)
    rn().rn_rotary(one.expand(1, 1, N, 2), None, theta, q_out=out)
    for at in (0, (1 << 28) - 50, (1 << 29) - 50, N - 100, 123456789):
        n = min(100, N - at)
        want = rn().rn_rotary(one.expand(1, 1, n, 2), None, theta, pos0=at)
        assert torch.equal(out[:, :, at:at + n], want), at
