"""The selective scan with infinite operands on the GPU: results are infinite, finite or NaN where the
float64 oracle's are, at state counts that do not fill a kernel's registers, channels that do not fill a
wave and tokens that do not fill a tile. Signs are chosen so that the formula adds no infinities of
different signs; decays are slow, so that none underflows (0 times infinity) over a segment."""
import numpy as np
import pytest
import torch

from oracle import scan as O
from tests.test_gpu_selective_scan import Batch, f64, rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


def positive(seed, lens, D, n, G, kind, packed, **kw):
    """A batch of positive values and slow decays."""
    b = Batch(seed, lens, D, n, G, kind, packed, **{"gate": False, **kw})
    for k in ("x", "dy", "B", "C", "state", "dstate", "skip"):
        t = getattr(b, k)
        if t is not None:
            setattr(b, k, t.abs() + 0.01)
    b.A = -b.A.abs() / n
    return b


def same_kinds(got, want):
    got, want = f64(got), np.asarray(want)
    return np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want)) and \
        np.array_equal(np.isneginf(got), np.isneginf(want))


STATES = [1, 3, 5, 7, 11, 13, 16, 20, 33]


@pytest.mark.parametrize("n", STATES)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,packed", [(40, False), (130, False), (130, True)])
def test_prompts(n, kind, N, packed):
    """An infinite input and an infinite raw step make the outputs of their channels infinite from there on."""
    b = positive(n + N, [N, 21], 70, n, 1, kind, packed)
    clean, _ = b.run()
    b.x, b.dt = b.x.clone(), b.dt.clone()
    b.x[0, 20, 5] = INF
    b.dt[0, 22, 69] = INF
    out, state = b.run(state_out=True)
    for i, at, _ in b.spans():
        want, last = O.selective_scan(**b.sequence(i, at))
        assert same_kinds(out[at], want) and same_kinds(state[i], last)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 20:N, 5] = bad[0, 22:N, 69] = True
    assert torch.isposinf(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("n", STATES)
def test_single_tokens_agree_with_prompts(n):
    b = positive(n, [12], 70, n, 1, torch.float32, False, pad=0)
    b.x, b.dt = b.x.clone(), b.dt.clone()
    b.x[0, 3, 5] = INF
    b.dt[0, 4, 69] = INF
    out, last = b.run(state_out=True)
    state, one = b.state.clone(), lambda t, i: t[..., i:i + 1, :]  # noqa: E731
    steps = [rn().rn_selective_scan_step(one(b.x, t), one(b.dt, t), b.A, one(b.B, t), one(b.C, t), state, b.skip, dt_bias=b.bias)
             for t in range(12)]
    assert same_kinds(torch.cat(steps, 1), f64(out)) and same_kinds(state, f64(last))
