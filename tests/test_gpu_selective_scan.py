"""The selective scan on the GPU against the float64 oracle.

Tolerances, in steps of 2^-24. The step D is off by at most 16 of itself (the sum of dt and the bias, the
exponential and the series of the softplus, for |dt + bias| up to 8). A decay exp(D A) has its exponent
off by 18 of |D A| and itself by 2; as |D A| exp(-|D A|) < 0.37, what it multiplies is off by 9 of
that. The token's own part is off by 19. So with H_t = exp(D_t A) H_{t-1} + |D_t x_t B_t| the sizes, a
token adds at most 32 H_t to what is off, which then decays with the state: W_t = exp(D_t A) W_{t-1} +
H_t. Cut into segments, a segment's decay has a sum of up to n steps as its exponent: 0.37 n more. The
output adds the states' products and the gate: (n states + 16) of the sum of sizes. Then half a step of
the output's type."""
import numpy as np
import pytest
import torch

from oracle import scan as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Batch:
    """Random sequences: padded with lengths, or packed with rows behind the last one."""

    def __init__(self, seed, lens, D, n, G=1, kind=torch.float32, packed=False, pad=3, gate=True, skip=True, bias=True,
                 start=True, view=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.packed, self.D, self.n, self.G = lens, packed, D, n, G
        rows = sum(lens) + pad if packed else max(max(lens), 1) + pad
        B = 1 if packed else len(lens)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        tok = lambda d: rnd(B, rows, d + 2 * view).to(kind).to(DEV)[..., view:d + view]  # noqa: E731
        self.x, self.z, self.dy = tok(D), tok(D) if gate else None, tok(D)
        self.dt = tok(D)
        heads = lambda: tok(G * n).unflatten(-1, (G, n)).transpose(1, 2)  # noqa: E731
        self.B, self.C = heads(), heads()
        self.A = (-torch.arange(1, n + 1) * torch.exp(rnd(D, n) * 0.3)).to(DEV)
        self.skip = rnd(D).to(DEV) if skip else None
        self.bias = (rnd(D) - 3).to(DEV) if bias else None
        self.state = rnd(len(lens), D, n).to(DEV) if start else None
        self.dstate = rnd(len(lens), D, n).to(DEV)
        self.kw = {}
        if packed:
            self.kw["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        else:
            self.kw["lengths"] = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def spans(self):
        at = 0
        for i, n in enumerate(self.lens):
            yield i, (0, slice(at, at + n)) if self.packed else (i, slice(0, n)), n
            at += n

    def rest(self, t):
        m = torch.ones(t.shape[:2], dtype=torch.bool, device=t.device)
        for _, at, _ in self.spans():
            m[at] = False
        return t[m]

    def run(self, softplus=True, **kw):
        return rn().rn_selective_scan_chunked(self.x, self.dt, self.A, self.B, self.C, self.skip, dt_bias=self.bias,
                                              softplus=softplus, z=self.z, state_in=self.state, **{**self.kw, **kw})

    def sequence(self, i, at):
        r, t = at
        return dict(x=f64(self.x[at]), dt=f64(self.dt[at]), A=f64(self.A), B=f64(self.B[r][:, t]), C=f64(self.C[r][:, t]),
                    skip=f64(self.skip), bias=f64(self.bias), z=None if self.z is None else f64(self.z[at]),
                    state=None if self.state is None else f64(self.state[i]))


def bounds(p, softplus):
    """(of the output before its rounding, of the final state) in steps: see above."""
    n, D = p["x"].shape
    A, G = p["A"], len(p["B"])
    v = p["dt"] + (0 if p["bias"] is None else p["bias"])
    step = np.logaddexp(v, 0) if softplus else v
    Bc, Cc = (np.abs(np.repeat(p[k], D // G, 0)).transpose(1, 0, 2) for k in "BC")
    H = np.zeros_like(A) if p["state"] is None else np.abs(p["state"])
    W = H.copy()
    y, c = np.zeros_like(p["x"]), 32 + 0.37 * n
    for t in range(n):
        a = np.exp(step[t][:, None] * A)
        H = a * H + np.abs(step[t] * p["x"][t])[:, None] * Bc[t]
        W = a * W + H
        y[t] = (Cc[t] * (c * W + (A.shape[1] + 16) * H)).sum(1)
    if p["skip"] is not None:
        y += 4 * np.abs(p["skip"] * p["x"])
    if p["z"] is not None:
        s = np.abs(p["z"] * O.sigmoid(p["z"]))
        y = y * s + (8 + 2 * np.abs(p["z"])) * np.abs(O.selective_scan(**{**p, "z": None}, softplus=softplus)[0]) * s
    return y * U, c * W * U


def check(b, out, state, softplus, kind):
    assert (b.rest(out) == 0).all()
    for i, at, _ in b.spans():
        p = b.sequence(i, at)
        want, h = O.selective_scan(softplus=softplus, **p)
        yb, hb = bounds(p, softplus)
        assert (np.abs(f64(out[at]) - want) <= yb + HALF[kind] * np.abs(want) + 1e-37).all(), i
        assert (np.abs(f64(state[i]) - h) <= hb + 1e-37).all(), i


SIZES = [([1], 1, 1, 1), ([16], 64, 16, 1), ([17, 0, 1], 65, 16, 1), ([15, 33], 6, 4, 3), ([5, 48], 130, 3, 2), ([40], 63, 8, 1),
         ([2, 3], 66, 12, 3), ([31], 20, 24, 2), ([20, 7], 64, 32, 1), ([18], 33, 33, 1), ([19, 1], 8, 64, 2), ([16, 16], 128, 2, 1),
         ([300], 5, 16, 1), ([200, 0, 129, 64], 70, 16, 1), ([260, 130], 4, 5, 2)]


@pytest.mark.parametrize("lens,D,n,G", SIZES)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [False, True])
def test_prompts(lens, D, n, G, kind, packed):
    for k, (kw, softplus) in enumerate([(dict(), True), (dict(gate=False, skip=False, start=False), True),
                                        (dict(view=1), True), (dict(bias=False, gate=False), False), (dict(view=2, skip=False), True)]):
        b = Batch(D * 3 + n + k, lens, D, n, G, kind, packed, **kw)
        if not softplus:
            b.dt = b.dt.abs() * 0.1            # steps as they are
        out, state = b.run(softplus, state_out=True)
        check(b, out, state, softplus, kind)


@pytest.mark.parametrize("D,n,G", [(1, 1, 1), (6, 4, 3), (65, 16, 1), (130, 3, 2), (64, 24, 1), (40, 64, 2), (1000, 8, 1)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_single_tokens(D, n, G, kind):
    for view in (0, 1):
        b = Batch(D + n, [1] * 5, D, n, G, kind, False, pad=0, view=view)
        state = b.state.clone()
        out = rn().rn_selective_scan_step(b.x, b.dt, b.A, b.B, b.C, state, b.skip, dt_bias=b.bias, z=b.z)
        check(b, out, state, True, kind)


def test_single_tokens_go_on_where_prompts_end():
    b = Batch(21, [90, 90], 70, 16, 2, torch.float32, False, pad=0)
    whole, last = b.run(state_out=True)
    cut = lambda t, a, e: t[..., a:e, :]  # noqa: E731
    _, state = rn().rn_selective_scan_chunked(*(cut(t, 0, 80) for t in (b.x, b.dt)), b.A, cut(b.B, 0, 80), cut(b.C, 0, 80),
                                              b.skip, dt_bias=b.bias, z=cut(b.z, 0, 80), state_in=b.state, state_out=True)
    outs = [rn().rn_selective_scan_step(*(cut(t, i, i + 1) for t in (b.x, b.dt)), b.A, cut(b.B, i, i + 1), cut(b.C, i, i + 1),
                                        state, b.skip, dt_bias=b.bias, z=cut(b.z, i, i + 1)) for i in range(80, 90)]
    for i, at, _ in b.spans():
        p = b.sequence(i, at)
        want, h = O.selective_scan(**p)
        yb, hb = bounds(p, True)
        assert (np.abs(f64(torch.cat(outs, 1)[i]) - want[80:]) <= yb[80:] + U * np.abs(want[80:])).all()
        assert (np.abs(f64(state[i]) - h) <= hb).all()
    assert np.abs(f64(last) - f64(state)).max() < 1e-4


def test_slots_in_place_and_skipped_sequences():
    for lens in ([5, 1, 0, 8], [200, 130, 0, 70]):
        b = Batch(3, lens, 40, 16, 1, torch.float32, True, start=False)
        pool = torch.randn(7, 40, 16, generator=torch.Generator().manual_seed(1)).to(DEV)
        before = pool.clone()
        slots = torch.tensor([6, 2, -1, 9], dtype=torch.int32, device=DEV)
        b.state = pool
        out, s = b.run(state_out=pool, slots=slots)
        assert s is pool
        b.state = torch.stack([before[int(i)] if 0 <= i < 7 else torch.zeros_like(before[0]) for i in slots])
        want, last = b.run(state_out=True)
        assert torch.equal(out, want) and torch.equal(pool[6], last[0]) and torch.equal(pool[2], last[1])
        for i in (0, 1, 3, 4, 5):
            assert torch.equal(pool[i], before[i])
    b = Batch(4, [1] * 4, 40, 16, 1, torch.float32, False, pad=0)
    before = pool.clone()
    out = rn().rn_selective_scan_step(b.x, b.dt, b.A, b.B, b.C, pool, b.skip, dt_bias=b.bias, z=b.z, slots=slots)
    assert (out[2:] == 0).all() and (out[:2] != 0).any()
    for i in (0, 1, 3, 4, 5):
        assert torch.equal(pool[i], before[i])
    assert not torch.equal(pool[6], before[6])


def test_rows_past_max_len_and_given_outputs():
    for packed in (False, True):
        b = Batch(8, [80, 200], 48, 16, 1, torch.bfloat16, packed)
        out = torch.full_like(b.x, 7.0)
        _, s1 = b.run(out=out, max_len=150, state_out=True)
        new, s2 = b.run(max_len=150, state_out=True)
        assert torch.equal(s1, s2)
        b.lens = [80, 150] if not packed else b.lens
        if packed:
            assert (out[0, 230:] == 7).all() and (new[0, 230:] == 0).all() and torch.equal(out[0, :230], new[0, :230])
        else:
            assert (b.rest(out) == 7).all() and (b.rest(new) == 0).all()
            assert torch.equal(out[0, :80], new[0, :80]) and torch.equal(out[1, :150], new[1, :150])


def test_values_that_are_not_finite_reach_later_tokens_of_their_channel_only():
    for N in (40, 400):
        b = Batch(4, [N], 72, 16, 1, torch.float32, False, pad=0)
        clean, _ = b.run()
        b.x = b.x.clone()
        b.x[0, 20, 5] = float("nan")
        out, state = b.run(state_out=True)
        bad = out.isnan()
        assert bad[0, 20:, 5].all() and not bad[0, :20].any() and state[0, 5].isnan().all()
        keep = torch.ones_like(bad)
        keep[0, 20:, 5] = False
        assert torch.equal(out[keep], clean[keep])
        b.B = b.B.clone()
        b.B[0, 0, 30, 3] = float("inf")
        out, _ = b.run()
        assert torch.equal(out[0, :20], clean[0, :20]) and not out[0, 30:].isfinite().any()


def test_steps_large_and_small():
    """Raw steps from -60 to 60: the softplus is the step itself at one end and its exponential at the
    other; decays reach 0 and 1."""
    b = Batch(6, [64], 64, 4, 1, torch.float32, False, pad=0, bias=False, start=True, gate=False)
    b.dt = torch.linspace(-60, 60, 64, device=DEV)[None, :, None].expand(1, 64, 64).contiguous()
    out, state = b.run(state_out=True)
    p = b.sequence(0, (0, slice(0, 64)))
    want, h = O.selective_scan(**p)
    yb, hb = bounds(p, True)
    # (the raw step's own rounding counts for more here: |dt| up to 60 of its exponential)
    assert (np.abs(f64(out[0]) - want) <= 8 * yb + U * np.abs(want) + 1e-37).all()
    assert (np.abs(f64(state[0]) - h) <= 8 * hb + 1e-37).all()


def test_cu_seqlens_that_make_no_sense_stay_inside_the_tensors():
    b = Batch(2, [300], 32, 16, 1, torch.float32, True, pad=0, start=False)
    x = b.x[:, 100:200]
    for cu in ([0, 90, 20, 60], [0, 1 << 30, -5, 100], [-7, 50, 50, 1 << 30], [100, 100, 0, 0]):
        out = torch.full((1, 300, 32), 7.0, device=DEV)
        rn().rn_selective_scan_chunked(x, b.dt[:, 100:200], b.A, b.B[:, :, 100:200], b.C[:, :, 100:200],
                                       cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), out=out[:, 100:200])
        assert (out[:, :100] == 7).all() and (out[:, 200:] == 7).all()


def test_steps_at_the_ends_of_the_type():
    """A token whose raw step is the type's lowest value or minus infinity changes no state (its step is
    zero); one with infinities or NaN reaches later tokens of its channel only."""
    low = torch.finfo(torch.bfloat16).min
    for N in (40, 400):
        b = Batch(14, [N], 72, 16, 1, torch.bfloat16, False, pad=0, gate=False, skip=False)
        b.dt = b.dt.clone()
        b.dt[0, 11] = low
        b.dt[0, 12] = float("-inf")
        out, state = b.run(state_out=True)
        assert out.isfinite().all() and state.isfinite().all()
        keep = [t for t in range(N) if t not in (11, 12)]
        cut = lambda t: t[..., keep, :].contiguous()  # noqa: E731
        rest, last = rn().rn_selective_scan_chunked(cut(b.x), cut(b.dt), b.A, cut(b.B), cut(b.C), dt_bias=b.bias, state_in=b.state,
                                                    state_out=True)
        assert np.abs(f64(state) - f64(last)).max() <= 1e-4 * np.abs(f64(last)).max()
        assert (np.abs(f64(cut(out)) - f64(rest)) <= 2.0 ** -7 * np.abs(f64(rest)) + 1e-4).all()
        b.dt[0, 20, 3], b.dt[0, 20, 4] = float("inf"), float("nan")
        bad, _ = b.run(state_out=True)
        assert torch.equal(bad[0, :20], out[0, :20]) and bad[0, 20:, 4].isnan().all()
        other = [c for c in range(72) if c not in (3, 4)]
        assert torch.equal(bad[0][:, other], out[0][:, other])
