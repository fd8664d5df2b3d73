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


# ---- gradients ------------------------------------------------------------------------------

def gradients(b, **kw):
    return rn().rn_selective_scan_backward(b.dy, b.x, b.dt, b.A, b.B, b.C, b.skip, dt_bias=b.bias, z=b.z, state_in=b.state,
                                           dstate_out=b.dstate, want_dstate_in=True, **{**b.kw, **kw})


def oracle_gradients(b):
    """The oracle's gradients in the calls' layouts, and zeros in rows of no sequence."""
    got = {k: np.zeros(b.x.shape) for k in ("dx", "ddt")}
    got.update({k: np.zeros(b.B.shape) for k in ("dB", "dC")})
    got["dstate_in"] = np.zeros(b.state.shape)
    with np.errstate(all="ignore"):
        for i, (r, t), _ in b.spans():
            w = O.selective_scan_backward(f64(b.dy[r, t]), dstate=f64(b.dstate[i]), **b.sequence(i, (r, t)))
            for k in ("dx", "ddt"):
                got[k][r, t] = w[k]
            for k in ("dB", "dC"):
                got[k][r][:, t] = w[k]
            got["dstate_in"][i] = w["dstate_in"]
            for k in ("dA", "dD", "ddt_bias"):
                got[k] = got.get(k, 0) + w[k]
    return got


# Tokens, channels and groups: pieces of one tile, and (150 blocks along the channels) of several. Channel 4 is never
# the one that lanes past its group repeat.
GRADS = [(1, 70, 1), (11, 70, 1), (13, 70, 1), (90, 70, 1), (251, 300, 150)]


@pytest.mark.parametrize("n", [5, 12, 16, 17, 32, 33])
@pytest.mark.parametrize("last,D,G", GRADS)
@pytest.mark.parametrize("packed", [False, True])
def test_an_infinite_last_input_reaches_its_channels_sums_alone(n, last, D, G, packed):
    """dD and the bias's gradient hold the last token's input: infinite there at any length, as they are elsewhere."""
    b = positive(n + last, [last, 13], D, n, G, torch.float32, packed)
    clean = gradients(b)
    b.x = b.x.clone()
    b.x[0, last - 1, 4] = INF
    got = gradients(b)
    others = [c for c in range(D) if c != 4]
    for k in ("dD", "ddt_bias"):
        assert torch.isposinf(got[k][4]) and torch.equal(got[k][others], clean[k][others]), k
    assert torch.equal(got["dA"], clean["dA"]) and torch.equal(got["dx"], clean["dx"])


@pytest.mark.parametrize("n", [4, 16, 24, 64])
@pytest.mark.parametrize("last,D,G", GRADS)
def test_an_infinite_gradient_of_the_last_state(n, last, D, G):
    b = positive(n + last, [last, 13], D, n, G, torch.float32, True)
    b.dstate[0, 4, n - 1] = INF
    got, want = gradients(b), oracle_gradients(b)
    for k, w in want.items():
        assert same_kinds(got[k], w), k


@pytest.mark.parametrize("n", [4, 16, 24, 64])
@pytest.mark.parametrize("last,D,G", GRADS)
def test_a_state_that_forgets_at_once(n, last, D, G):
    """A of minus infinity: its decay is 0, and only the step's own gradient (0 times A) is NaN. The operands
    being positive, the sums of sizes that rounding counts in are the gradients themselves, times at
    most the tokens: 360 2^-24 of them for each."""
    b = positive(n + last, [last, 13], D, n, G, torch.float32, True)
    b.A[4, 1] = -INF
    got, want = gradients(b), oracle_gradients(b)
    for k, w in want.items():
        if "ddt" in k:
            assert same_kinds(got[k], w), k
        else:
            assert (np.abs(f64(got[k]) - w) <= 360 * 2.0 ** -24 * (last + 13) * np.abs(w)).all(), k


@pytest.mark.parametrize("n", [1, 3, 5, 11, 13, 16, 20, 33, 40])
@pytest.mark.parametrize("last,D,G", GRADS[1:])
@pytest.mark.parametrize("where", ["x", "dt", "dy"])
def test_an_infinite_operand_of_one_channel(n, last, D, G, where):
    """Whatever states the registers hold past the n: infinities of an input, a raw step or an output's gradient."""
    b = positive(n + last, [last, 13], D, n, G, torch.float32, True)
    t = getattr(b, where).clone()
    t[0, last // 2, 4] = INF
    setattr(b, where, t)
    got, want = gradients(b), oracle_gradients(b)
    for k, w in want.items():
        assert same_kinds(got[k], w), k


@pytest.mark.parametrize("n", [4, 12, 16, 24, 48])
@pytest.mark.parametrize("last,D,G", GRADS[1:])
@pytest.mark.parametrize("where", ["B", "C", "state", "dstate"])
def test_an_infinite_operand_of_all_channels_or_of_the_last(n, last, D, G, where):
    """Lanes past a group's channels work on its last one, or on B and C, too: sums over channels leave them out."""
    b = positive(n + last, [last, 13], D, n, G, torch.float32, True)
    t = getattr(b, where).clone()
    if where in "BC":
        t[0, 0, last // 2, 1] = INF
    else:
        t[0, D - 1, 1] = INF
    setattr(b, where, t)
    got, want = gradients(b), oracle_gradients(b)
    for k, w in want.items():
        assert same_kinds(got[k], w), k
