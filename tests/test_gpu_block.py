"""The operators around retention used together, on streams, and in captured graphs."""
import numpy as np
import pytest
import torch

from oracle import block as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


class Layer:
    """norm -> projections -> rotary -> linear attention -> group norm -> out projection, in
    float32: the tests below run it as a prompt, token by token, and backward through its norm."""

    def __init__(self, seed, D=96, H=4, Hk=2, dk=16, dv=24):
        g = torch.Generator().manual_seed(seed)
        self.H, self.Hk, self.dk, self.dv = H, Hk, dk, dv
        cols = H * dk + Hk * dk + H * dv + H
        self.w = (torch.randn(D, cols, generator=g) / D ** 0.5).to(DEV)
        self.wo = (torch.randn(H * dv, D, generator=g) / (H * dv) ** 0.5).to(DEV)
        self.nw, self.nb = (torch.randn(D, generator=g) * 0.1 + 1).to(DEV), (torch.randn(D, generator=g) * 0.1).to(DEV)
        self.theta, self.m = rn().rn_rotary_frequencies(8, kind="by_parts", factor=2.0, length=64)

    def split(self, p):
        """Views of the projection [B, N, cols] as heads, and the decays."""
        H, Hk, dk, dv = self.H, self.Hk, self.dk, self.dv
        q, k, v, g = p.split([H * dk, Hk * dk, H * dv, H], -1)
        heads = lambda t, h: t.unflatten(-1, (h, -1)).transpose(1, 2)  # noqa: E731
        return heads(q, H), heads(k, Hk), heads(v, H), torch.nn.functional.logsigmoid(g + 2).transpose(1, 2)

    def __call__(self, x, r, state, pos, step):
        n, h = rn().rn_layernorm(x, self.nw, self.nb, residual=r)
        q, k, v, g = self.split(n @ self.w)
        rn().rn_rotary(q, k, self.theta, pos=pos, half=True, magnitude=self.m, q_out=q, k_out=k)
        if step:
            o = rn().rn_linear_attention_step(q, k, v, g, state, qk_scale=0.25)
        else:
            o, _ = rn().rn_linear_attention_chunked(q, k, v, g, state_in=state, state_out=state, qk_scale=0.25)
        o = rn().rn_groupnorm_gate(o.contiguous())
        return o.transpose(1, 2).flatten(2) @ self.wo, h

    def oracle(self, x, r, pos):
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        n, h = K.layernorm(x, self.nw, self.nb, 1e-5, r)
        q, k, v, g = (f(t) for t in self.split(torch.tensor(n) @ self.w.double().cpu()))
        q = K.rotary(q, self.theta, pos, True, magnitude=self.m)
        k = K.rotary(k, self.theta, pos, True, magnitude=self.m)
        o, S = zip(*(K.linear_attention(q[b], k[b], v[b], g[b], 0.25) for b in range(len(q))))
        y = np.stack([K.layernorm(a)[0] for a in o])
        return y.transpose(0, 2, 1, 3).reshape(len(q), y.shape[2], -1) @ f(self.wo), h, np.stack(S)


def data(seed, B, N, D=96):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, N, D, generator=g).to(DEV) for _ in range(2))


def close(a, b):
    """Float32 through about ten operators on sums of at most 100 terms: 1e-4 of the largest
    value (1e-4 is the framework's own bound for float32 retention; group norm divides by the
    spread of 24 values, whose smallest of a few hundred rows may be a tenth of the mean)."""
    a = a.double().cpu().numpy() if isinstance(a, torch.Tensor) else a
    return np.abs(a - b).max() <= 1e-4 * np.abs(b).max()


def test_prompt_and_single_tokens_against_the_oracle():
    L = Layer(1)
    B, N, P = 2, 90, 80
    x, r = data(2, B, N)
    first = torch.tensor([5, 1000], device=DEV)
    state = torch.zeros(B, L.H, L.dk, L.dv, device=DEV)
    cut = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    y, h = L(cut(x, 0, P), cut(r, 0, P), state, first, False)
    ys, hs = [y], [h]
    for t in range(P, N):
        y, h = L(cut(x, t, t + 1), cut(r, t, t + 1), state, first + t, True)
        ys.append(y)
        hs.append(h)
    want, hw, S = L.oracle(x, r, np.arange(N)[None] + first.cpu().numpy()[:, None])
    assert close(torch.cat(ys, 1), want) and close(torch.cat(hs, 1), hw) and close(state, S)


def test_norm_backward_joins_the_residual_stream():
    """d loss / d x of loss = sum(dy norm(x + r)) + sum(dh (x + r)) through autograd in float64."""
    x, r = data(3, 2, 33)
    dy, dh = data(4, 2, 33)
    L = Layer(1)
    _, h = rn().rn_layernorm(x, L.nw, L.nb, residual=r)
    got = rn().rn_layernorm_backward(dy, h, L.nw, dsum=dh)
    p = [t.double().cpu().requires_grad_() for t in (x, L.nw, L.nb)]
    s = p[0] + r.double().cpu()
    y = torch.nn.functional.layer_norm(s, (96,), p[1], p[2])
    ((y * dy.double().cpu()).sum() + (s * dh.double().cpu()).sum()).backward()
    for a, b in zip((got["dx"], got["dweight"], got["dbias"]), p):
        assert close(a, b.grad.numpy())


def test_rotary_and_norm_feed_the_retention_layer():
    """A pre-norm retention block: norm, then the library's gated layer, residual joined by the
    next norm; equal to the same calls on a normalised tensor from torch's own float64."""
    import workloads as W
    w = W.Workload("t", "chunkwise", B=1, H=2, N=70, d_k=64, d_v=64, dtype="bf16", chunk=32, gn=True, gate=True, qkv_std=0.25, seed=3)
    x = W.make_layer_inputs(w, 128)
    X = x["x"].to(DEV)
    n = rn().rn_layernorm(X)
    ref = torch.nn.functional.layer_norm(X.double(), (128,)).bfloat16()
    assert (n != ref).float().mean() < 0.02 and (n.float() - ref.float()).abs().max() <= 2.0 ** -7 * 4   # a step apart at most
    ws = [x[k].to(DEV) for k in ("w_q", "w_k", "w_v", "w_g", "w_o")]
    y, _ = rn().rn_msr_layer_forward(n, *ws, x["gamma"], x["theta"], 2, 64, 64, 32)
    n2, s = rn().rn_layernorm(y, residual=X)
    want = torch.nn.functional.layer_norm((y.double() + X.double()), (128,))
    assert torch.equal(s, (y.float() + X.float()).bfloat16())
    assert (n2.double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() * 1.01


def calls(x, r, dy, qkv, pool, slots, theta):
    """One call of every operator on the given tensors, results in a list."""
    out, s = rn().rn_layernorm(x, residual=r)
    got = [out, s] + list(rn().rn_layernorm_backward(dy, s).values())
    q, k, v, g = qkv
    a, b = rn().rn_rotary(q, k, theta, pos0=3)
    o, S = rn().rn_linear_attention_chunked(a, b, v, g, state_out=True)
    got += [a, b, o, S]
    got.append(rn().rn_linear_attention_step(a[:, :, :1], b[:, :, :1], v[:, :, :1], g[:, :, :1], pool, slots=slots))
    return got


def setup(seed, N=1500):
    g = torch.Generator().manual_seed(seed)
    x, r, dy = (torch.randn(70, 256, generator=g).bfloat16().to(DEV) for _ in range(3))
    q, k, v = (torch.randn(1, 2, N, 64, generator=g).bfloat16().to(DEV) for _ in range(3))
    dec = (-torch.rand(1, 2, N, generator=g) * 0.1).to(DEV)
    return x, r, dy, (q, k, v, dec), torch.randn(3, 2, 64, 64, generator=g).to(DEV), torch.tensor([1], dtype=torch.int32, device=DEV)


def test_other_streams_give_the_same_bits():
    """Calls on two side streams at once, each on tensors of its own, waiting on nothing but
    their own inputs."""
    theta = 10000.0 ** (-np.arange(32) / 32)
    sets = [setup(s) for s in (5, 6)]
    want = [calls(*(t.clone() if torch.is_tensor(t) else t for t in s), theta) for s in sets]
    pools = [s[4].clone() for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for rep in range(3):
        for i, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                s[4].copy_(pools[i])
                got[i] = calls(*s, theta)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_captured_and_replayed_with_changing_inputs():
    """One graph of all operators, replayed on new inputs with eager work between the replays;
    every replay against the eager results."""
    theta = 10000.0 ** (-np.arange(32) / 32)
    s = setup(7)
    x, r, dy, qkv, pool, slots = s
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(*s, theta)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*s, theta)
    for seed in (8, 9, 10):
        n = setup(seed)
        for a, b in zip((x, r, dy, *qkv, pool), (*n[:3], *n[3], n[4])):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        after = pool.clone()
        want = calls(*n, theta)                       # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, want)) and torch.equal(after, n[4])


def test_tensors_of_another_device_than_the_current_one(monkeypatch):
    """The binding makes the tensors' GPU current for the call (here it is told that another is)."""
    from linear_recurrent_sequence_rn_amd import block_ops
    s = setup(11)
    theta = 10000.0 ** (-np.arange(32) / 32)
    copy = [t.clone() if torch.is_tensor(t) else t for t in s]
    want = calls(*copy, theta)
    monkeypatch.setattr(block_ops, "_current_device", lambda: 7)
    got = calls(*s, theta)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.cuda.current_device() == 0


def test_group_norm_of_more_rows_than_one_grid_axis_takes():
    """2^26 + 9 rows of 4 values: rows from all over the call equal those of short calls, bit by bit."""
    N = (1 << 26) + 9
    x = torch.randn(1, 1, N, 4, generator=torch.Generator(DEV).manual_seed(33), device=DEV).bfloat16()
    out = rn().rn_groupnorm_gate(x, out=torch.zeros_like(x))
    for at in (0, (1 << 25) - 50, (1 << 26) - 50, N - 100, 12345678):
        n = min(100, N - at)
        assert torch.equal(out[:, :, at:at + n], rn().rn_groupnorm_gate(x[:, :, at:at + n].contiguous())), at
