"""RMS norm, short convolution and selective scan as a block uses them together: prompts, single tokens,
gradients, streams, captured graphs, another device."""
import numpy as np
import pytest
import torch

from oracle import scan as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


def f64(t):
    return t.double().cpu().numpy()


class Block:
    """norm with the residual's sum -> projection to x and z -> convolution -> projections to dt, B and C ->
    gated scan -> projection back, in float32."""

    def __init__(self, seed, D=48, E=96, n=16, K=4, G=2):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.E, self.n, self.G, self.K = E, n, G, K
        self.nw = (r(D) * 0.1 + 1).to(DEV)
        self.win = (r(D, 2 * E) / D ** 0.5).to(DEV)
        self.cw, self.cb = (r(E, K) / K ** 0.5).to(DEV), (r(E) * 0.1).to(DEV)
        self.wx = (r(E, E + 2 * G * n) / E ** 0.5).to(DEV)
        self.bias = (r(E) * 0.5 - 3).to(DEV)
        self.A = (-torch.arange(1, n + 1) * torch.exp(r(E, n) * 0.1)).to(DEV)
        self.skip = (r(E) * 0.1 + 1).to(DEV)
        self.wo = (r(E, D) / E ** 0.5).to(DEV)

    def heads(self, t):
        return t.unflatten(-1, (self.G, self.n)).transpose(1, 2)

    def states(self, S):
        return torch.zeros(S, self.K - 1, self.E, device=DEV), torch.zeros(S, self.E, self.n, device=DEV)

    def __call__(self, x, r, conv, state, step=False, **batch):
        """(out, sum); the states are updated in place."""
        y, h = rn().rn_rmsnorm(x, self.nw, residual=r)
        u, z = (y @ self.win).split(self.E, -1)
        if step:
            u = rn().rn_short_conv_step(u, self.cw, self.cb, conv, silu=True)
        else:
            u, _ = rn().rn_short_conv(u, self.cw, self.cb, silu=True, state_in=conv, state_out=conv, **batch)
        dt, B, C = (u @ self.wx).split([self.E, self.G * self.n, self.G * self.n], -1)
        B, C = self.heads(B), self.heads(C)
        if step:
            o = rn().rn_selective_scan_step(u, dt, self.A, B, C, state, self.skip, dt_bias=self.bias, z=z)
        else:
            o, _ = rn().rn_selective_scan_chunked(u, dt, self.A, B, C, self.skip, dt_bias=self.bias, z=z, state_in=state,
                                                  state_out=state, **batch)
        return o @ self.wo, h

    def oracle(self, x, r):
        """(out, sum, final states) of one sequence [n, D]."""
        y, h = O.rmsnorm(x, f64(self.nw), 1e-5, r)
        u, z = np.split(y @ f64(self.win), 2, -1)
        u, conv = O.short_conv(u, f64(self.cw), f64(self.cb), True)
        p = u @ f64(self.wx)
        m = self.G * self.n
        heads = lambda t: t.reshape(len(t), self.G, self.n).transpose(1, 0, 2)  # noqa: E731
        o, S = O.selective_scan(u, p[:, :self.E], f64(self.A), heads(p[:, self.E:self.E + m]), heads(p[:, self.E + m:]),
                                f64(self.skip), f64(self.bias), True, z)
        return o @ f64(self.wo), h, conv, S

    def parts(self):
        return {"nw": self.nw, "win": self.win, "cw": self.cw, "cb": self.cb, "wx": self.wx, "bias": self.bias, "A": self.A,
                "skip": self.skip, "wo": self.wo}

    def backward(self, x, r, dout, dh):
        """Gradients of sum(dout out) + sum(dh sum) from zero states, the calls' own backwards joined."""
        E, m = self.E, self.G * self.n
        y, h = rn().rn_rmsnorm(x, self.nw, residual=r)
        xz = y @ self.win
        u0, z = xz.split(E, -1)
        u, _ = rn().rn_short_conv(u0, self.cw, self.cb, silu=True)
        p = u @ self.wx
        dt, B, C = p.split([E, m, m], -1)
        B, C = self.heads(B), self.heads(C)
        o, _ = rn().rn_selective_scan_chunked(u, dt, self.A, B, C, self.skip, dt_bias=self.bias, z=z)
        flat = lambda t: t.flatten(0, 1)  # noqa: E731
        g = {"wo": flat(o).t() @ flat(dout)}
        dxz, dp = torch.empty_like(xz), torch.empty_like(p)
        dB, dC = self.heads(dp[..., E:E + m]), self.heads(dp[..., E + m:])
        s = rn().rn_selective_scan_backward(dout @ self.wo.t(), u, dt, self.A, B, C, self.skip, dt_bias=self.bias, z=z,
                                            ddt=dp[..., :E], dB=dB, dC=dC, dz=dxz[..., E:])
        g.update(A=s["dA"], skip=s["dD"], bias=s["ddt_bias"], wx=flat(u).t() @ flat(dp))
        c = rn().rn_short_conv_backward(s["dx"] + dp @ self.wx.t(), u0, self.cw, self.cb, silu=True, dx=dxz[..., :E])
        g.update(cw=c["dweight"], cb=c["dbias"], win=flat(y).t() @ flat(dxz))
        n = rn().rn_rmsnorm_backward(dxz @ self.win.t(), h, self.nw, dsum=dh)
        g.update(nw=n["dweight"], x=n["dx"])
        return g


def data(seed, B, N, D=48):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, N, D, generator=g).to(DEV) for _ in range(2)]


def close(a, b, bound=1e-4):
    """Float32 through about ten operators on sums of at most 200 terms: 1e-4 of the largest value, as
    the blocks of linear attention are held to."""
    a = f64(a) if isinstance(a, torch.Tensor) else a
    return np.abs(a - b).max() <= bound * np.abs(b).max()


def test_prompt_and_single_tokens_against_the_oracle():
    L = Block(1)
    B, N, P = 2, 150, 140
    x, r = data(2, B, N)
    conv, state = L.states(B)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    ys, hs = zip(L(cut(x, 0, P), cut(r, 0, P), conv, state), *(L(cut(x, t, t + 1), cut(r, t, t + 1), conv, state, True) for t in range(P, N)))
    want = [L.oracle(f64(x[b]), f64(r[b])) for b in range(B)]
    y, h = torch.cat(ys, 1), torch.cat(hs, 1)
    for b, (wy, wh, wc, wS) in enumerate(want):
        assert close(y[b], wy) and close(h[b], wh) and close(conv[b], wc) and close(state[b], wS)


def test_packed_prompts_equal_padded_ones():
    L = Block(3)
    lens = [40, 1, 0, 97, 3]
    x, r = data(4, 5, 97)
    conv, state = L.states(5)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    y, _ = L(x, r, conv, state, lengths=n)
    px, pr = (torch.cat([t[i, :m] for i, m in enumerate(lens)])[None].contiguous() for t in (x, r))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    c2, s2 = L.states(5)
    z, _ = L(px, pr, c2, s2, cu_seqlens=cu, max_len=97)
    want = torch.cat([y[i, :m] for i, m in enumerate(lens)])
    assert close(z[0], f64(want)) and close(c2, f64(conv)) and close(s2, f64(state))


def test_gradients_against_differences_of_the_oracle():
    """The loss's slope along each gradient, by central differences in float64 (off by 1e-6 of the
    loss's size over 1e-4, and by the third derivative): within 1e-3 of the gradient's size there."""
    L = Block(5)
    x, r = data(6, 1, 40)
    dout, dh = data(7, 1, 40)
    g = L.backward(x, r, dout, dh)
    par = L.parts()

    def loss():
        out, h, _, _ = L.oracle(X, f64(r[0]))
        return (out * f64(dout[0])).sum() + (h * f64(dh[0])).sum()
    X = f64(x[0])
    for name in [*par, "x"]:
        d = f64(g[name] if name != "x" else g["x"][0])
        d = d / np.linalg.norm(d)
        keep = X.copy() if name == "x" else par[name].double().cpu()
        e = 1e-4 * np.linalg.norm(keep) / keep.size ** 0.5 if name == "x" else 1e-4 * float(keep.norm()) / keep.numel() ** 0.5
        values = []
        for sign in (1, -1):
            if name == "x":
                X = keep + sign * e * d
            else:
                setattr(L, name, keep + sign * e * torch.tensor(d))
            values.append(loss())
        if name == "x":
            X = keep
        else:
            setattr(L, name, par[name])
        slope = float((f64(g[name] if name != "x" else g["x"][0]) * d).sum())
        assert abs((values[0] - values[1]) / (2 * e) - slope) <= 1e-3 * abs(slope), name


def setup(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)  # noqa: E731
    E, n, T = 136, 16, 700
    return {"x": r(70, 256), "res": r(70, 256), "dy": r(70, 256), "u": r(1, T, E), "dt": r(1, T, E), "z": r(1, T, E), "du": r(1, T, E),
            "B": r(1, 1, T, n), "C": r(1, 1, T, n), "A": (-torch.rand(E, n, generator=g) * 4).to(DEV),
            "bias": (torch.randn(E, generator=g) - 3).to(DEV), "w": torch.randn(E, 4, generator=g).to(DEV),
            "conv": r(3, 3, E), "state": torch.randn(3, E, n, generator=g).to(DEV),
            "cu": torch.tensor([0, 100, 101, 650], dtype=torch.int32, device=DEV), "slots": torch.tensor([2], dtype=torch.int32, device=DEV)}


def calls(s):
    """One call of every operator; results in a list."""
    m = rn()
    q, h, sc = m.rn_rmsnorm(s["x"], residual=s["res"], out_dtype=torch.float8_e4m3fn, group=64)
    got = [q.float(), h, sc] + list(m.rn_rmsnorm_backward(s["dy"], h).values())
    u, c = m.rn_short_conv(s["u"], s["w"], s["bias"], silu=True, cu_seqlens=s["cu"], state_in=s["conv"], state_out=True)
    got += [u, c] + list(m.rn_short_conv_backward(s["du"], s["u"], s["w"], s["bias"], silu=True, cu_seqlens=s["cu"],
                                                  want_dstate_in=True).values())
    scan = (s["A"], s["B"], s["C"])
    o, S = m.rn_selective_scan_chunked(u, s["dt"], *scan, dt_bias=s["bias"], z=s["z"], cu_seqlens=s["cu"], state_in=s["state"], state_out=True)
    got += [o, S] + list(m.rn_selective_scan_backward(s["du"], u, s["dt"], *scan, dt_bias=s["bias"], z=s["z"], cu_seqlens=s["cu"],
                                                      state_in=s["state"], want_dstate_in=True).values())
    one = lambda t: t[..., :1, :]  # noqa: E731
    got.append(m.rn_short_conv_step(one(s["u"]), s["w"], None, s["conv"], slots=s["slots"]))
    got.append(m.rn_selective_scan_step(one(s["u"]), one(s["dt"]), s["A"], one(s["B"]), one(s["C"]), s["state"], slots=s["slots"]))
    return got + [s["conv"], s["state"]]


def clone(s):
    return {k: t.clone() for k, t in s.items()}


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_streams_give_the_same_bits():
    """Calls on two side streams at once, each on tensors of its own."""
    sets = [setup(i) for i in (5, 6)]
    want = [[t.clone() for t in calls(clone(s))] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for rep in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = calls(clone(sets[i]))
        torch.cuda.synchronize()
        for i in range(2):
            assert same(got[i], want[i])


def test_captured_and_replayed_with_changing_inputs():
    """One graph of all operators, replayed on new inputs with eager work between the replays; every
    replay against the eager results."""
    s = setup(7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(clone(s))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(s)
    for seed in (8, 9, 10):
        n = setup(seed)
        for k in s:
            s[k].copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        want = calls(n)                               # eager work between the replays
        torch.cuda.synchronize()
        assert same(first, want)


def test_two_graphs_share_a_workspace():
    """Two captured graphs of the scan and its gradients on one workspace, replayed in turn."""
    m = rn()
    sets = [setup(i) for i in (11, 12)]
    need = max(m.rn_selective_scan_workspace_bytes(sets[0]["u"], sets[0]["A"], sets[0]["B"]),
               m.rn_selective_scan_backward_workspace_bytes(sets[0]["u"], sets[0]["A"], sets[0]["B"]))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def run(s, ws=None):
        o, S = m.rn_selective_scan_chunked(s["u"], s["dt"], s["A"], s["B"], s["C"], z=s["z"], state_out=True, workspace=ws)
        return [o, S] + list(m.rn_selective_scan_backward(s["du"], s["u"], s["dt"], s["A"], s["B"], s["C"], z=s["z"], workspace=ws).values())
    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(run(s, ws))
        graphs.append(g)
    for rep in range(3):
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """The binding makes the tensors' GPU current for the call (here it is told that another is)."""
    from linear_recurrent_sequence_rn_amd import block_ops
    s = setup(13)
    want = [t.clone() for t in calls(clone(s))]
    monkeypatch.setattr(block_ops, "_current_device", lambda: 7)
    got = calls(clone(s))
    assert same(got, want) and torch.cuda.current_device() == 0


def test_arguments_that_do_not_fit_are_refused():
    m = rn()
    s = setup(14)
    u, dt, A, B, C = s["u"], s["dt"], s["A"], s["B"], s["C"]
    bad = [lambda: m.rn_rmsnorm(s["x"], residual=s["res"][:3]), lambda: m.rn_rmsnorm(s["x"], scale_out=s["bias"]),
           lambda: m.rn_rmsnorm(s["x"], s["bias"]), lambda: m.rn_rmsnorm(s["x"].half()),
           lambda: m.rn_rmsnorm(s["x"], out_dtype=torch.float8_e4m3fn, group=48), lambda: m.rn_rmsnorm(s["x"], group=32),
           lambda: m.rn_rmsnorm(s["x"], out=s["x"], sum_out=s["x"]), lambda: m.rn_rmsnorm_backward(s["dy"][:1], s["x"]),
           lambda: m.rn_short_conv(u, s["w"][:3]), lambda: m.rn_short_conv(u, s["w"].bfloat16()), lambda: m.rn_short_conv(u[0], s["w"]),
           lambda: m.rn_short_conv(u, s["w"], out=u), lambda: m.rn_short_conv(u, s["w"], state_in=s["state"]),
           lambda: m.rn_short_conv(u, s["w"], cu_seqlens=s["cu"].long()), lambda: m.rn_short_conv(u, s["w"], max_len=701),
           lambda: m.rn_short_conv(u, torch.zeros(136, 9, device=DEV)), lambda: m.rn_short_conv(u.transpose(1, 2), s["w"]),
           lambda: m.rn_short_conv(u, s["w"], slots=s["slots"], state_out=True),
           lambda: m.rn_short_conv_step(u, s["w"], None, s["conv"]), lambda: m.rn_short_conv_backward(s["dy"], u, s["w"]),
           lambda: m.rn_selective_scan_chunked(u, dt, A, B, C[..., :8]), lambda: m.rn_selective_scan_chunked(u, dt.float(), A, B, C),
           lambda: m.rn_selective_scan_chunked(u, dt, A.bfloat16(), B, C), lambda: m.rn_selective_scan_chunked(u, dt, A, B, C, out=dt),
           lambda: m.rn_selective_scan_chunked(u, dt, A, B.expand(1, 3, 700, 16), C.expand(1, 3, 700, 16)),
           lambda: m.rn_selective_scan_chunked(u, dt, A, B, C, state_in=s["state"][:, :5]),
           lambda: m.rn_selective_scan_chunked(u, dt, A, B, C, workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
           lambda: m.rn_selective_scan_step(u, dt, A, B, C, s["state"]),
           lambda: m.rn_selective_scan_backward(s["du"], u, dt, A, B, C, dz=u), lambda: m.rn_selective_scan_backward(s["du"], u, dt, A, B, C, dx=u),
           lambda: m.rn_selective_scan_backward(s["du"], u, dt, A, B, C, dB=dt)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, m.RnError)):
            f()
            raise AssertionError(i)
