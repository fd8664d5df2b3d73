"""Elements more than 2^31 from a tensor's start: the same bits as for the same values side by side."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FAR = (1 << 31) + 64


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.mem_get_info(0)[0] < 96 << 30:
        pytest.skip("needs 96 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def far(t):
    """t [2, ...] with its second row FAR elements behind its first one."""
    v = torch.empty(FAR + t[1].numel(), dtype=t.dtype, device=DEV).as_strided(t.shape, (FAR, *t.stride()[1:]))
    return v.copy_(t)


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().to(DEV)


def far_pool(t):
    """t [2, ...] as the first and the last state of a pool of more than 2^31 elements."""
    slots = FAR // t[0].numel() + 2
    pool = torch.empty((slots, *t.shape[1:]), dtype=t.dtype, device=DEV)
    pool[0], pool[-1] = t[0], t[1]
    return pool, torch.tensor([0, slots - 1], dtype=torch.int32, device=DEV)


def test_convolution():
    x, dy = rand(1, 2, 40, 72), rand(2, 2, 40, 72)
    w, bias = rand(3, 72, 4).float(), rand(4, 72).float()
    want, last = rn().rn_short_conv(x, w, bias, silu=True, state_out=True)
    fx, fdy, out, dx = (far(t) for t in (x, dy, torch.zeros_like(x), torch.zeros_like(x)))
    rn().rn_short_conv(fx, w, bias, silu=True, out=out)
    assert torch.equal(out, want)
    need = rn().rn_short_conv_backward(dy, x, w, bias, silu=True)
    got = rn().rn_short_conv_backward(fdy, fx, w, bias, silu=True, dx=dx)
    assert all(torch.equal(got[k], need[k]) for k in need)
    pool, slots = far_pool(last)
    one = rn().rn_short_conv_step(x[:, :1], w, bias, last, silu=True)
    assert torch.equal(rn().rn_short_conv_step(x[:, :1], w, bias, pool, silu=True, slots=slots), one)
    assert torch.equal(pool[0], last[0]) and torch.equal(pool[-1], last[1])


@pytest.mark.parametrize("n", [16, 40])
def test_scan(n):
    x, dt, z, dy = (rand(i, 2, 200, 72) for i in range(4))
    B, C = rand(5, 2, 1, 200, n), rand(6, 2, 1, 200, n)
    A = -rand(7, 72, n).float().abs()
    want, last = rn().rn_selective_scan_chunked(x, dt, A, B, C, z=z, state_out=True)
    fx, fdt, fz, fdy, out, dx, ddt, dz = (far(t) for t in (x, dt, z, dy, *[torch.zeros_like(x)] * 4))
    fB, fC, dB, dC = (far(t) for t in (B, C, torch.zeros_like(B), torch.zeros_like(B)))
    rn().rn_selective_scan_chunked(fx, fdt, A, fB, fC, z=fz, out=out)
    assert torch.equal(out, want)
    need = rn().rn_selective_scan_backward(dy, x, dt, A, B, C, z=z)
    got = rn().rn_selective_scan_backward(fdy, fx, fdt, A, fB, fC, z=fz, dx=dx, ddt=ddt, dz=dz, dB=dB, dC=dC)
    assert all(torch.equal(got[k], need[k]) for k in need)
    pool, slots = far_pool(last)
    rows = [t[:, :1] for t in (x, dt)], [t[:, :, :1] for t in (B, C)]
    one = rn().rn_selective_scan_step(*rows[0], A, *rows[1], last)
    assert torch.equal(rn().rn_selective_scan_step(*rows[0], A, *rows[1], pool, slots=slots), one)
    assert torch.equal(pool[0], last[0]) and torch.equal(pool[-1], last[1])


def test_norm():
    x, dy = rand(1, 2, 200), rand(2, 2, 200)
    w = rand(3, 200).float()
    fx, fdy = far(x), far(dy)
    assert torch.equal(rn().rn_rmsnorm(fx, w), rn().rn_rmsnorm(x, w))
    got, need = rn().rn_rmsnorm_backward(fdy, fx, w), rn().rn_rmsnorm_backward(dy, x, w)
    assert all(torch.equal(got[k], need[k]) for k in need)
