"""The RMS norm's values in 8 bits are its float32 output over the scale, rounded once: nothing is lost on the
way, whatever lies beside a border between two values."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def quotient(y, scale, group):
    """y / scale in float32, rounded once (a float64 quotient of two float32 rounded to float32 is that)."""
    each = scale.repeat_interleave(group, -1)[..., :y.shape[-1]] if group else scale[..., None]
    return (y.double() / each.double()).float()


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,group", [(3000, 4096, 0), (3000, 4096, 128), (40000, 256, 32), (5001, 1537, 64)])
def test_values_of_eight_bits_are_the_quotient_rounded_once(kind, dt, rows, d, group):
    import linear_recurrent_sequence_rn_amd as rn
    g = torch.Generator(DEV).manual_seed(rows + d + group)
    x, r = (torch.randn(rows, d, generator=g, device=DEV).to(dt) for _ in range(2))
    w = torch.randn(d, generator=g, device=DEV) * 0.2 + 1
    y, _ = rn.rn_rmsnorm(x, w, residual=r, out_dtype=torch.float32)
    out, _, scale = rn.rn_rmsnorm(x, w, residual=r, out_dtype=kind, group=group)
    q = quotient(y, scale, group)
    want = q.to(kind) if kind is torch.float8_e4m3fn else q.round().to(kind)
    assert int((out.float() != want.float()).sum()) == 0


@pytest.mark.parametrize("kind", [torch.float8_e4m3fn, torch.int8])
def test_rows_under_small_scales(kind):
    """Rows from 1e-37 to 1: their scales reach down to the smallest one and are no powers of two."""
    import linear_recurrent_sequence_rn_amd as rn
    g = torch.Generator(DEV).manual_seed(4)
    x = torch.randn(400, 512, generator=g, device=DEV) * torch.logspace(-37, 0, 400, device=DEV)[:, None]
    y = rn.rn_rmsnorm(x, None, 1.0, out_dtype=torch.float32)
    out, scale = rn.rn_rmsnorm(x, None, 1.0, out_dtype=kind)
    q = quotient(y, scale, 0)
    want = q.to(kind) if kind is torch.float8_e4m3fn else q.round().to(kind)
    assert int((out.float() != want.float()).sum()) == 0
