"""Root-mean-square norm on the GPU against the float64 oracle.

Tolerances. A row's sum of squares adds positive terms: at most 16 in a lane and 10 levels of a tree, each
rounding 2^-24 of it, so rstd is within (26 / 2 + 4) 2^-24; h, the two products and a scale add a few
more: R = 24 steps of 2^-24 of the value. Then the output's own rounding, half a step of its type."""
import numpy as np
import pytest
import torch

from oracle import scan as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
R = 24 * U
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy()


def normal(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def near(got, want, half):
    want = np.asarray(want)
    return (np.abs(f64(got) - want) <= (half + R) * np.abs(want) + 1e-37).all()


SIZES = [(1, 1), (3, 7), (2, 64), (5, 128), (17, 129), (4, 255), (3, 256), (9, 512), (33, 1000), (2, 1025), (7, 2048),
         (3, 4097), (2, 8192), (3, 12289), (2, 16384)]


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_forward(rows, d, kind):
    g = torch.Generator().manual_seed(rows * 31 + d)
    x, r, w = normal(g, rows, d, dtype=kind, std=2.0), normal(g, rows, d, dtype=kind), normal(g, d)
    for other in (torch.float32, torch.bfloat16):
        out = rn().rn_rmsnorm(x, out_dtype=other)
        assert out.dtype == other and near(out, O.rmsnorm(f64(x))[0], HALF[other])
        out, s = rn().rn_rmsnorm(x, w, 1e-3, residual=r, out_dtype=other)
        y, h = O.rmsnorm(f64(x), f64(w), 1e-3, f64(r))
        assert near(out, y, HALF[other])
        assert torch.equal(s, (x.float() + r.float()).to(kind))


def check_held(out, scale, y, kind, group):
    """A value in 8 bits is off by half its step: 2^-4 of it in e4m3, or half of the smallest step
    (2^-9) of the scale; half the scale in int8."""
    most = 448.0 if kind is torch.float8_e4m3fn else 127.0
    want = O.scales(y, most, group)
    assert (np.abs(f64(scale) - want) <= R * want).all()
    each = O.spread(want, y.shape[-1], group)
    off = np.abs(out.float().double().cpu().numpy() * O.spread(f64(scale), y.shape[-1], group) - y)
    half = np.maximum(np.abs(y) * 2.0 ** -4, each * 2.0 ** -10) if most == 448.0 else each * 0.5
    assert (off <= half * (1 + 4 * R) + 2 * R * np.abs(y) + 1e-37).all()


@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
def test_eight_bits(rows, d, group, kind):
    g = torch.Generator().manual_seed(rows + d * 7)
    for dt in (torch.bfloat16, torch.float32):
        x, r, w = normal(g, rows, d, dtype=dt, std=2.0), normal(g, rows, d, dtype=dt), normal(g, d)
        out, scale = rn().rn_rmsnorm(x, w, out_dtype=kind, group=group)
        assert out.dtype == kind and scale.shape == ((rows, -(-d // group)) if group else (rows,))
        check_held(out, scale, O.rmsnorm(f64(x), f64(w))[0], kind, group)
        out, s, scale = rn().rn_rmsnorm(x, residual=r, out_dtype=kind, group=group)
        check_held(out, scale, O.rmsnorm(f64(x), None, 1e-5, f64(r))[0], kind, group)
        assert torch.equal(s, (x.float() + r.float()).to(dt))


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("group", [0, 32])
def test_eight_bits_of_rows_at_the_ends_of_the_range(kind, group):
    """Zeros give zeros under the smallest scale; a NaN or infinity makes its scale NaN (the row's root
    mean square is not finite then, so every scale of the row); other rows are as they are alone."""
    x = torch.zeros(6, 96)
    x[1] = torch.randn(96, generator=torch.Generator().manual_seed(1))
    x[2, 40] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 1e-30
    x[5, 7] = 3.0
    x = x.to(DEV)
    out, scale = rn().rn_rmsnorm(x, eps=1e-6, out_dtype=kind, group=group)
    v, s = out.float().cpu(), scale.cpu().reshape(6, -1)
    assert (v[0] == 0).all() and (s[0] == 2.0 ** -126).all()
    assert s[2].isnan().all() and s[3].isnan().any()
    if kind is torch.float8_e4m3fn:
        assert v[2].isnan().all()
    else:
        assert (v[2] == 0).all()
    for i in (1, 4, 5):
        a, b = rn().rn_rmsnorm(x[i:i + 1].contiguous(), eps=1e-6, out_dtype=kind, group=group)
        assert torch.equal(a.float(), out[i:i + 1].float()) and torch.equal(b, scale[i:i + 1])
        check_held(out[i:i + 1], scale[i:i + 1], O.rmsnorm(f64(x[i:i + 1]), eps=1e-6)[0], kind, group)
    if group:                                # columns of zeros beside others: the smallest scale
        assert (s[5, 1:] == 2.0 ** -126).all() and s[5, 0] > 1e-3


@pytest.mark.parametrize("d", [96, 101])
def test_strided_rows_and_in_place(d):
    g = torch.Generator().manual_seed(d)
    big = normal(g, 7, 2 * d + 3, dtype=torch.bfloat16)
    x, r = big[:, 1:d + 1], big[:, d + 2:2 * d + 2]
    want, h = rn().rn_rmsnorm(x.contiguous(), residual=r.contiguous())
    got, s = rn().rn_rmsnorm(x, residual=r)
    assert torch.equal(got, want) and torch.equal(s, h)
    a, b = x.contiguous(), r.contiguous()
    got, s = rn().rn_rmsnorm(a, residual=b, sum_out=b, out=a)
    assert got is a and s is b and torch.equal(a, want) and torch.equal(b, h)
    held = torch.zeros(7, 2 * d, dtype=torch.int8, device=DEV)
    q, sc = rn().rn_rmsnorm(x, out=held[:, 3:d + 3])
    q2, sc2 = rn().rn_rmsnorm(x.contiguous(), out_dtype=torch.int8)
    assert torch.equal(q, q2) and torch.equal(sc, sc2)
    assert (held[:, :3] == 0).all() and (held[:, d + 3:] == 0).all()


@pytest.mark.parametrize("rows,d", SIZES + [(300, 96), (1000, 2048)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_backward(rows, d, kind):
    """dx: 40 steps of 2^-24 of its terms' sizes (rstd as above, the mean of products with 16 + 10 + 3
    roundings); dw: a lane's rows, 32 sums and 32 more of at most (rows / 4 + 64) roundings."""
    g = torch.Generator().manual_seed(rows * 13 + d)
    x, dy, dh, w = normal(g, rows, d, dtype=kind, std=2.0), normal(g, rows, d, dtype=kind), normal(g, rows, d, dtype=kind), normal(g, d)
    for weight, dsum in ((w, dh), (None, None)):
        got = rn().rn_rmsnorm_backward(dy, x, weight, 1e-4, dsum=dsum)
        dx, dw = O.rmsnorm_backward(f64(dy), f64(x), None if weight is None else f64(weight), 1e-4, None if dsum is None else f64(dsum))
        X = f64(x)
        rs = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + 1e-4)
        gw = np.abs(f64(dy) * (1.0 if weight is None else f64(weight)))
        size = rs * (gw + np.abs(X) * rs * (gw * np.abs(X) * rs).mean(-1, keepdims=True)) + (0 if dsum is None else np.abs(f64(dsum)))
        assert (np.abs(f64(got["dx"]) - dx) <= 40 * U * size + HALF[kind] * np.abs(dx)).all()
        big = np.abs(f64(dy) * X * rs).sum(0)
        assert (np.abs(f64(got["dweight"]) - dw) <= (24 + 64 + rows / 4) * U * big).all()


def test_backward_in_place_without_weight_gradient_and_repeatable():
    g = torch.Generator().manual_seed(5)
    x, dy, dh, w = (normal(g, 400, 520, dtype=torch.bfloat16) for _ in range(3)), None, None, normal(g, 520)
    x, dy, dh = x
    want = rn().rn_rmsnorm_backward(dy, x, w, dsum=dh)
    again = rn().rn_rmsnorm_backward(dy, x, w, dsum=dh)
    assert torch.equal(want["dx"], again["dx"]) and torch.equal(want["dweight"], again["dweight"])
    for k in range(3):
        t = [x.clone(), dy.clone(), dh.clone()]
        got = rn().rn_rmsnorm_backward(t[1], t[0], w, dsum=t[2], dx=t[k], want_dweight=False)
        assert "dweight" not in got and got["dx"] is t[k] and torch.equal(t[k], want["dx"])


def test_rows_of_large_calls_equal_those_of_small_ones():
    """Calls past the last-level cache take other loads; the values are the same bits."""
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.randn(20000, 4096, generator=g, device=DEV).bfloat16()
    out, scale = rn().rn_rmsnorm(x, out_dtype=torch.float8_e4m3fn, group=128)
    o2, s, sc2 = rn().rn_rmsnorm(x, residual=x, out_dtype=torch.float8_e4m3fn)
    for a in (0, 7777, 19900):
        part = x[a:a + 100].contiguous()
        p, ps = rn().rn_rmsnorm(part, out_dtype=torch.float8_e4m3fn, group=128)
        assert torch.equal(p.float(), out[a:a + 100].float()) and torch.equal(ps, scale[a:a + 100])
        p, q, ps = rn().rn_rmsnorm(part, residual=part, out_dtype=torch.float8_e4m3fn)
        assert torch.equal(p.float(), o2[a:a + 100].float()) and torch.equal(ps, sc2[a:a + 100]) and torch.equal(q, s[a:a + 100])
