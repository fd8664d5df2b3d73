"""Gradients of the selective scan on the GPU against the float64 oracle and against differences of the
forward call.

Tolerances, in steps of 2^-24, as for the forward call (tests/test_gpu_selective_scan.py): with H_t the
states' sizes, c = 32 + 0.37 n and W_t = exp(D_t A) W_{t-1} + H_t, a state is off by at most c W_t. The
gradient g_t of a state runs the same recurrence backward, from the sizes |C_t dy_t| (dy, with the gate, off
by 8 + 2 |z|): with G_t its sizes and V_t = G_t + exp(D_{t+1} A) V_{t+1}, it is off by at most (c + 8 + 2 max
|z|) V_t. Every gradient sums products of these: with the sizes W and V in the place of the values, a
product of two is off by twice that, and the sums (states, 64 channels and their blocks, a piece's tokens and
the pieces) add at most 160 roundings: K = 2 (c + 16) + 160 steps of the sum of sizes (|z| <= 4 here).
Then half a step of the output's type."""
import numpy as np
import pytest
import torch

from oracle import scan as O
from tests.test_gpu_selective_scan import HALF, U, Batch, f64, rn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def batch(*args, **kw):
    b = Batch(*args, **kw)
    if b.z is not None:
        b.z.clamp_(-4, 4)
    return b


def run(b, softplus=True, **kw):
    return rn().rn_selective_scan_backward(b.dy, b.x, b.dt, b.A, b.B, b.C, b.skip, dt_bias=b.bias, softplus=softplus, z=b.z,
                                           state_in=b.state, **{**b.kw, **kw})


def sizes(p, dy, ds, softplus):
    """The sums of sizes behind each gradient of one sequence."""
    n, D = p["x"].shape
    A, G = p["A"], len(p["B"])
    v = p["dt"] + (0 if p["bias"] is None else p["bias"])
    step = np.logaddexp(v, 0) if softplus else v
    slope = O.sigmoid(v) if softplus else np.ones_like(v)
    Bc, Cc = (np.abs(np.repeat(p[k], D // G, 0)).transpose(1, 0, 2) for k in "BC")
    x, dz = np.abs(p["x"]), np.abs(dy)
    if p["z"] is not None:
        s = O.sigmoid(p["z"])
        # the gate's slope s (1 + z (1 - s)) adds terms that cancel near z = -1.28, where its roundings
        # stay those of the terms: 3 of s and 3 of z s (1 - s)
        out = np.abs(dy) * (s + np.abs(p["z"]) * s * (1 - s))
        dz, dy = out, np.abs(dy * p["z"] * s)
    dy = np.abs(dy)
    H = np.zeros_like(A) if p["state"] is None else np.abs(p["state"])
    W, Ws = H.copy(), []
    P = []
    for t in range(n):
        a = np.exp(step[t][:, None] * A)
        P.append(a * W)
        H = a * H + (step[t] * x[t])[:, None] * Bc[t]
        W = a * W + H
        Ws.append(W)
    Gs = np.abs(ds)
    V = Gs.copy()
    m = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dA=np.zeros_like(A), dB=np.zeros((G, n, A.shape[1])), dC=np.zeros((G, n, A.shape[1])))
    y = np.zeros_like(x)
    for t in reversed(range(n)):
        a = np.exp(step[t][:, None] * A)
        Gs = Gs + Cc[t] * dy[t][:, None]
        V = V + Gs
        m["dC"][:, t] = (Ws[t] * dy[t][:, None]).reshape(G, -1, A.shape[1]).sum(1)
        m["dB"][:, t] = (V * (step[t] * x[t])[:, None]).reshape(G, -1, A.shape[1]).sum(1)
        du = (V * Bc[t]).sum(1)
        m["dx"][t] = du * step[t]
        m["ddt"][t] = (du * x[t] + (V * P[t] * np.abs(A)).sum(1)) * slope[t]
        m["dA"] += V * P[t] * step[t][:, None]
        y[t] = (Cc[t] * Ws[t]).sum(1)
        Gs, V = a * Gs, a * V
    if p["skip"] is not None:
        m["dx"] += np.abs(p["skip"]) * dy
        m["dD"] = (dy * x).sum(0)
        y += np.abs(p["skip"]) * x
    if p["z"] is not None:
        m["dz"] = dz * y
    m["ddt_bias"] = m["ddt"].sum(0)
    m["dstate_in"] = V
    return m


def check(b, got, softplus, kind, dstate):
    tokens = ("dx", "ddt") + (("dz",) if b.z is not None else ())
    total, room = {}, {}
    for name in tokens:
        assert (b.rest(got[name]) == 0).all(), name
    for name in ("dB", "dC"):
        assert (b.rest(got[name].transpose(1, 2)) == 0).all(), name
    for i, at, n in b.spans():
        p = b.sequence(i, at)
        dy, ds = f64(b.dy[at]), np.zeros((b.D, b.n)) if dstate is None else f64(dstate[i])
        want = O.selective_scan_backward(dy, softplus=softplus, dstate=ds, **p)
        size = sizes(p, dy, ds, softplus)
        k = (2 * (32 + 0.37 * n + 16) + 160) * U
        for name in tokens:
            assert (np.abs(f64(got[name][at]) - want[name]) <= k * size[name] + HALF[kind] * np.abs(want[name]) + 1e-37).all(), (name, i)
        for name in ("dB", "dC"):
            g = f64(got[name][at[0]][:, at[1]])
            assert (np.abs(g - want[name]) <= k * size[name] + HALF[kind] * np.abs(want[name]) + 1e-37).all(), (name, i)
        if "dstate_in" in got:
            assert (np.abs(f64(got["dstate_in"][i]) - want["dstate_in"]) <= k * size["dstate_in"] + 1e-37).all(), i
        for name in ("dA", "dD", "ddt_bias"):
            if name in got:
                total[name] = total.get(name, 0) + want[name]
                room[name] = room.get(name, 0) + k * size[name]
    for name in total:
        assert (np.abs(f64(got[name]) - total[name]) <= room[name] + U * np.abs(total[name]) + 1e-37).all(), name


SIZES = [([1], 1, 1, 1), ([16], 64, 16, 1), ([17, 0, 1], 65, 16, 1), ([15, 33], 6, 4, 3), ([5, 48], 130, 3, 2), ([40], 63, 8, 1),
         ([2, 3], 66, 12, 3), ([31], 20, 24, 2), ([20, 70], 64, 32, 1), ([18, 40], 33, 33, 1), ([19, 1], 8, 64, 2), ([130, 16], 128, 2, 1),
         ([300], 5, 16, 1), ([200, 0, 129, 64], 70, 16, 1), ([64, 65, 128], 140, 16, 2), ([260, 130], 4, 5, 2)]


@pytest.mark.parametrize("lens,D,n,G", SIZES)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients(lens, D, n, G, kind, packed):
    for k, (kw, softplus) in enumerate([(dict(), True), (dict(gate=False, skip=False, start=False), True),
                                        (dict(view=1), True), (dict(bias=False, gate=False), False)]):
        b = batch(D * 3 + n + k, lens, D, n, G, kind, packed, **kw)
        if not softplus:
            b.dt = b.dt.abs() * 0.1            # steps as they are
        dstate = b.dstate if k != 1 else None
        got = run(b, softplus, dstate_out=dstate, want_dstate_in=k != 1)
        assert ("dz" in got) == (b.z is not None) and ("dD" in got) == (b.skip is not None)
        assert ("ddt_bias" in got) == (b.bias is not None) and ("dstate_in" in got) == (k != 1)
        check(b, got, softplus, kind, dstate)


def test_differences_of_the_forward_call():
    """The loss's change along random directions, each input by itself, over 2e: the loss is a sum of
    about 2e4 products off by 1e-6 each at random (1e-4 of a loss of about 1e2, over e = 0.01), and the third
    derivative counts e^2: within 2e-2 of the gradient's size along that direction."""
    b = batch(77, [90, 33], 70, 16, 2, torch.float32, True, pad=0)
    got = run(b, dstate_out=b.dstate, want_dstate_in=True)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", skip="dD", bias="ddt_bias", z="dz", state="dstate_in")

    def loss():
        out, last = b.run(state_out=True)
        return float((out.double() * b.dy).sum() + (last.double() * b.dstate).sum())
    for name, g in names.items():
        keep, grad = getattr(b, name), got[g].double()
        d = grad / grad.norm()
        e = 0.01 * float(keep.double().norm()) / keep.numel() ** 0.5
        setattr(b, name, (keep + e * d).float())
        up = loss()
        setattr(b, name, (keep - e * d).float())
        down = loss()
        setattr(b, name, keep)
        slope = float((grad * d).sum())
        assert abs((up - down) / (2 * e) - slope) <= 2e-2 * abs(slope) + 2e-2, name


def test_given_outputs_keep_rows_of_no_sequence():
    for packed in (False, True):
        b = batch(8, [80, 200], 48, 16, 1, torch.bfloat16, packed)
        new = run(b, max_len=150)
        both = torch.full((*b.x.shape[:2], 96), 7.0, dtype=torch.bfloat16, device=DEV)       # dx and dz as halves of one tensor
        heads = torch.full((*b.x.shape[:2], 32), 7.0, dtype=torch.bfloat16, device=DEV)
        dB, dC = (t.unflatten(-1, (1, 16)).transpose(1, 2) for t in heads.split(16, -1))
        got = run(b, max_len=150, dx=both[..., :48], dz=both[..., 48:], dB=dB, dC=dC)
        assert (new["ddt"] == got["ddt"]).all() and torch.equal(new["dA"], got["dA"])
        m = torch.zeros(b.x.shape[:2], dtype=torch.bool, device=DEV)
        if packed:
            m[0, :230] = True
        else:
            m[0, :80] = m[1, :150] = True
        for name, t in (("dx", both[..., :48]), ("dz", both[..., 48:]), ("dB", dB.transpose(1, 2)), ("dC", dC.transpose(1, 2))):
            w = new[name] if name in ("dx", "dz") else new[name].transpose(1, 2)
            assert (t[~m] == 7).all() and (w[~m] == 0).all() and torch.equal(t[m], w[m]), name


def test_the_same_bits_every_time_and_in_any_workspace():
    b = batch(9, [300, 150], 200, 16, 1, torch.bfloat16, True)
    need = rn().rn_selective_scan_backward_workspace_bytes(b.x, b.A, b.B, cu_seqlens=b.kw["cu_seqlens"])
    want = run(b, dstate_out=b.dstate, want_dstate_in=True)
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        got = run(b, dstate_out=b.dstate, want_dstate_in=True, workspace=ws)
        assert all(torch.equal(want[k], got[k]) for k in want)


def test_cu_seqlens_that_make_no_sense_stay_inside_the_tensors():
    b = batch(2, [300], 32, 16, 1, torch.float32, True, pad=0, start=False)
    cut = lambda t: t[..., 100:200, :]  # noqa: E731
    for cu in ([0, 90, 20, 60], [0, 1 << 30, -5, 100], [-7, 50, 50, 1 << 30], [100, 100, 0, 0]):
        big = {k: torch.full((1, 300, 32), 7.0, device=DEV) for k in ("dx", "ddt", "dz")}
        heads = {k: torch.full((1, 1, 300, 16), 7.0, device=DEV) for k in ("dB", "dC")}
        rn().rn_selective_scan_backward(cut(b.dy), cut(b.x), cut(b.dt), b.A, cut(b.B), cut(b.C), z=cut(b.z),
                                        cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                                        **{k: cut(t) for k, t in {**big, **heads}.items()})
        for t in (*big.values(), *heads.values()):
            assert (t[..., :100, :] == 7).all() and (t[..., 200:, :] == 7).all()


@pytest.mark.parametrize("n", [12, 16, 32, 33])
@pytest.mark.parametrize("last", [1, 8, 11, 90])
@pytest.mark.parametrize("packed", [False, True])
def test_an_infinite_last_input_leaves_the_decays_gradients(n, last, packed):
    """dA holds g_t a_t h_{t-1} D_t, which the input of a sequence's last token is in nowhere."""
    b = batch(n + last, [last, 13], 70, n, 1, torch.float32, packed)
    clean = run(b)
    b.x = b.x.clone()
    b.x[0, last - 1, 5] = float("inf")
    got = run(b)
    assert torch.equal(got["dA"], clean["dA"]) and torch.equal(got["dx"], clean["dx"])
    assert not got["ddt"][0, last - 1, 5].isfinite()
