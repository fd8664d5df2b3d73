"""Linear attention with a decay per head and token on the GPU against the float64 oracle.

Tolerances. u = 2^-24. With M = the same recurrence on |q|, |k|, |v| and E = the largest sum of
decays a token sees (sum over s <= t of the decay from s to t, at most the tokens in sight), a
float32 result is off by at most (3 E + d_k + 64) u M: each token adds three roundings to what
it finds, weighted by its decay; the sum over d_k, the waves and the segments adds d_k + 32, the
exponentials 32. A bf16 result adds half a step of its value, h = 2^-8. With matrix products in
bf16 the scores and the state's copy are rounded once: h M more; and since these roundings are
independent of each other and at most h/sqrt(3) in the mean square (as is that of the output),
the whole output's relative 2-norm error stays under sqrt(2) h / sqrt(3) = 0.0032."""
import numpy as np
import pytest
import torch

from oracle import block as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
H16 = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rn():
    import linear_recurrent_sequence_rn_amd as m
    return m


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def heads(gen, B, H, N, d, dt, token_major):
    shape = (B, N, H, d) if token_major else (B, H, N, d)
    x = torch.randn(shape, generator=gen).to(dt).to(DEV)
    return x.transpose(1, 2) if token_major else x


def inputs(B, H, Hq, Hk, Hv, N, dk, dv, kind, seed, token_major=False, fade=4.0, resets=0.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (heads(g, B, h, N, d, DT[kind], token_major) for h, d in ((Hq, dk), (Hk, dk), (Hv, dv)))
    dec = torch.nn.functional.logsigmoid(torch.randn(B, H, N, generator=g) + 2) / fade
    dec[torch.rand(B, H, N, generator=g) < resets] = -float("inf")
    return q, k, v, dec.to(DEV)


def reach(g):
    """The largest sum of decays a token sees, [H, n] -> number."""
    a, e, m = np.exp(np64(g)), 0.0, 1.0
    for t in range(a.shape[1]):
        e = e * a[:, t] + 1
        m = max(m, float(e.max()))
    return m


def check_sequence(out, state, q, k, v, g, scale, s0, mfma=False):
    """One sequence's outputs [H, n, dv] and final state (or None) against the oracle."""
    dk = q.shape[-1]
    o, S = K.linear_attention(q, k, v, g, scale, s0)
    mo, mS = K.linear_attention(q.abs(), k.abs(), v.abs(), g, abs(scale), None if s0 is None else s0.abs())
    c = (3 * reach(g) + dk + 64) * U
    h = torch.finfo(out.dtype).eps / 2 if out.dtype == torch.bfloat16 else 0.0
    tol = c * mo + 1.01 * h * np.abs(o) + (1.02 * H16 * mo if mfma else 0) + 1e-30
    off = np.abs(np64(out) - o)
    assert (off <= tol).all(), f"outputs: {(off / tol).max()} of the tolerance at {np.unravel_index((off / tol).argmax(), off.shape)}"
    if mfma and o.size > 2000:
        assert np.linalg.norm(np64(out) - o) <= 0.0032 * np.linalg.norm(o)
    if state is not None:
        off = np.abs(np64(state) - S)
        tol = c * mS + 1e-30
        assert (off <= tol).all(), f"state: {(off / tol).max()} of the tolerance at {np.unravel_index((off / tol).argmax(), off.shape)}"


def uses_mfma(kind, od, dk, dv, generic):
    return kind == "bf16" and od == torch.bfloat16 and not generic and dk % 8 == 0 and dv % 8 == 0


SHAPES = [  # B, H, Hq, Hk, Hv, N, dk, dv
    (1, 1, 1, 1, 1, 1, 1, 1), (2, 3, 3, 1, 3, 5, 3, 7), (1, 2, 2, 2, 2, 64, 64, 64), (1, 2, 1, 1, 2, 65, 64, 128),
    (2, 4, 4, 2, 2, 130, 128, 128), (1, 3, 3, 3, 1, 63, 48, 81), (1, 2, 2, 2, 2, 200, 256, 512), (1, 1, 1, 1, 1, 17, 255, 65),
    (3, 2, 2, 2, 2, 1, 128, 128), (1, 2, 2, 2, 2, 700, 16, 40), (1, 1, 1, 1, 1, 1000, 128, 64), (1, 4, 2, 4, 1, 129, 80, 96),
    (2, 2, 2, 2, 2, 96, 192, 256), (1, 1, 1, 1, 1, 300, 8, 8)]


@pytest.mark.parametrize("kind,out_kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,H,Hq,Hk,Hv,N,dk,dv", SHAPES)
def test_padded_batches(kind, out_kind, B, H, Hq, Hk, Hv, N, dk, dv):
    od = DT[out_kind]
    for tm, fade, resets, start in ((False, 4.0, 0.0, False), (True, 16.0, 0.02, True)):
        q, k, v, g = inputs(B, H, Hq, Hk, Hv, N, dk, dv, kind, B * 1000 + N + dk, tm, fade, resets)
        s0 = torch.randn(B, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(1)) if start else None
        scale = dk ** -0.5
        out, S = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=scale, state_in=s0, state_out=True, out_dtype=od)
        assert out.dtype == od and out.shape == (B, H, N, dv) and S.shape == (B, H, dk, dv)
        for b in range(B):
            check_sequence(out[b], S[b], q[b], k[b], v[b], g[b], scale, None if s0 is None else s0[b],
                           uses_mfma(kind, od, dk, dv, False))
        gen, S2 = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=scale, state_in=s0, state_out=True, out_dtype=od,
                                                   force_generic=True)
        for b in range(B):
            check_sequence(gen[b], S2[b], q[b], k[b], v[b], g[b], scale, None if s0 is None else s0[b])
        drop, none = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=scale, state_in=s0, out_dtype=od)
        assert none is None and torch.equal(drop, out)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lens,N", [([0, 1, 64, 65, 200], 200), ([700, 3, 0, 1300], 1300), ([-5, 4000, 17], 130)])
def test_lengths(kind, lens, N):
    """Ragged padded batch: lengths clamped to [0, N]; rows behind stay as they were."""
    B, H, dk, dv = len(lens), 2, 32, 48
    q, k, v, g = inputs(B, H, 2, 1, 2, N, dk, dv, kind, 7)
    n = [min(max(x, 0), N) for x in lens]
    for b in range(B):                                    # nothing behind a sequence is read
        for t in (q, k, v):
            t[b, :, n[b]:] = float("nan")
        g[b, :, n[b]:] = float("nan")
    s0 = torch.randn(B, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(2))
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = torch.full((B, H, N, dv), 7.0, dtype=DT[kind], device=DEV)
    _, S = rn().rn_linear_attention_chunked(q, k, v, g, lengths=ln, state_in=s0, state_out=True, out=out)
    new, _ = rn().rn_linear_attention_chunked(q, k, v, g, lengths=ln, state_in=s0)
    for b in range(B):
        assert (out[b, :, n[b]:] == 7.0).all() and (new[b, :, n[b]:] == 0.0).all()
        assert torch.equal(out[b, :, :n[b]], new[b, :, :n[b]])
        if n[b] == 0:
            assert torch.equal(S[b], s0[b])
        else:
            check_sequence(out[b, :, :n[b]], S[b], q[b, :, :n[b]], k[b, :, :n[b]], v[b, :, :n[b]], g[b, :, :n[b]], 1.0, s0[b],
                           kind == "bf16")
    _, Z = rn().rn_linear_attention_chunked(q, k, v, g, lengths=ln, state_out=True)
    for b in range(B):
        if n[b] == 0:
            assert int(torch.count_nonzero(Z[b])) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lens,rest", [([1], 0), ([5, 64, 0, 1, 130], 9), ([900, 2, 1500, 33], 700)])
def test_packed_batches_and_slots(kind, lens, rest):
    """Packed sequences with states in a pool: slots in any order, one sequence without a slot;
    the pool's other states and the rows behind the last sequence keep their bits."""
    S, T = len(lens), sum(lens) + rest
    H, Hq, Hk, Hv, dk, dv = 4, 2, 1, 4, 64, 64
    q, k, v, g = inputs(1, H, Hq, Hk, Hv, T, dk, dv, kind, 11, True)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    e = sum(lens)
    for t in (q, k, v, g):
        t[:, :, e:] = float("nan")
    pool = torch.randn(S + 3, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    before = pool.clone()
    order = np.random.default_rng(4).permutation(S + 3)[:S].astype(np.int32)
    if S > 1:
        order[1] = -1
    if S > 3:
        order[3] = S + 3                                   # outside the pool
    slots = torch.tensor(order, device=DEV)
    out = torch.full((1, H, T, dv), 7.0, dtype=DT[kind], device=DEV)
    rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, max_len=max(lens), state_in=pool, state_out=pool,
                                     slots=slots, out=out)
    assert (out[:, :, e:] == 7.0).all()
    new, _ = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, state_in=before, slots=slots)
    assert (new[:, :, e:] == 0.0).all() and new.stride(1) == dv
    used = set()
    for s, n in enumerate(lens):
        a, b = int(cu[s]), int(cu[s + 1])
        slot = int(order[s])
        has = 0 <= slot < S + 3
        used |= {slot} if has else set()
        s0 = before[slot] if has else None
        if n == 0:
            continue
        args = (q[0, :, a:b], k[0, :, a:b], v[0, :, a:b], g[0, :, a:b], 1.0, s0, kind == "bf16")
        check_sequence(out[0, :, a:b], pool[slot] if has else None, *args)
        check_sequence(new[0, :, a:b], None, *args)
    for i in range(S + 3):
        if i not in used or lens[list(order).index(i)] == 0:
            assert torch.equal(pool[i], before[i])


def test_cut_and_disordered_cu_seqlens_stay_inside():
    """max_len below a sequence's length cuts it; entries outside [0, T] or out of order are
    clamped, so that no call reaches outside its tensors."""
    H, dk, dv, T = 2, 64, 64, 300
    q, k, v, g = inputs(1, H, H, H, H, T, dk, dv, "bf16", 12, True)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device=DEV)
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, max_len=150, state_out=True)
    check_sequence(out[0, :, :150], S[0], q[0, :, :150], k[0, :, :150], v[0, :, :150], g[0, :, :150], 1.0, None, True)
    assert (out[0, :, 150:200] == 0).all()
    guard = torch.full((T + 200, H, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    o = guard[100:100 + T].transpose(0, 1)[None]
    bad = torch.tensor([-50, 1 << 30, 20, 40, -(1 << 30), 310], dtype=torch.int32, device=DEV)
    for generic in (True, False):
        rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=bad, out=o, state_out=True, force_generic=generic)
    torch.cuda.synchronize()
    assert (guard[:100] == 7.0).all() and (guard[100 + T:] == 7.0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_constant_decay_through_a_zero_stride_is_retention(kind):
    """One decay per head, repeated along the tokens by a stride of 0, equals retention with
    theta = 0, both within their float32 bounds of the same numbers."""
    B, H, N, d = 2, 3, 150, 32
    q, k, v, _ = inputs(B, H, H, H, H, N, d, d, kind, 13)
    gamma = np.array([1.0, 0.97, 0.5], dtype=np.float32)
    g = torch.tensor(np.log(gamma.astype(np.float64)), dtype=torch.float32, device=DEV)[None, :, None].expand(B, H, N)
    s0 = torch.randn(B, H, d, d, device=DEV, generator=torch.Generator(DEV).manual_seed(5))
    a, S = rn().rn_linear_attention_chunked(q, k, v, g, state_in=s0, state_out=True, out_dtype=torch.float32)
    b, R = rn().rn_retention_chunkwise(q, k, v, gamma, np.zeros(16), 32, state_in=s0, state_out=True, out_dtype=torch.float32)
    for i in range(B):
        check_sequence(a[i], S[i], q[i], k[i], v[i], g[i], 1.0, s0[i])
        scale = np.abs(np64(R[i])).max()
        assert np.abs(np64(S[i] - R[i])).max() <= 1e-4 * scale and (a[i] - b[i]).abs().max() <= 1e-4 * b[i].abs().max()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["q", "k", "v", "g"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_values_reach_only_later_tokens(kind, where, bad):
    """A NaN or infinity at token 100 leaves the tokens before it, and the other sequence, as
    they are without it."""
    B, H, N, dk, dv = 2, 2, 200, 64, 64
    q, k, v, g = inputs(B, H, H, H, H, N, dk, dv, kind, 14)
    clean, C = rn().rn_linear_attention_chunked(q, k, v, g, state_out=True)
    t = {"q": q, "k": k, "v": v, "g": g}[where]
    t[(1, 0, 100) if where == "g" else (1, 0, 100, 5)] = bad
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, state_out=True)
    assert torch.equal(out[0], clean[0]) and torch.equal(S[0], C[0]) and torch.equal(out[1, 1], clean[1, 1])
    assert torch.equal(out[1, 0, :100], clean[1, 0, :100])
    o, s = K.linear_attention(q[1], k[1], v[1], g[1])
    assert np.array_equal(np.isfinite(np64(out[1])), np.isfinite(o))
    assert np.array_equal(np.isfinite(np64(S[1])), np.isfinite(s))


def test_every_token_reset_and_strong_decays():
    """Decays of exactly 0 (each token sees itself alone) and very strong ones."""
    q, k, v, g = inputs(1, 2, 2, 2, 2, 150, 64, 64, "bf16", 15)
    s0 = torch.randn(1, 2, 64, 64, device=DEV, generator=torch.Generator(DEV).manual_seed(6))
    for val in (-float("inf"), -1e30, -80.0, -20.0, 0.0):
        g.fill_(val)
        out, S = rn().rn_linear_attention_chunked(q, k, v, g, state_in=s0, state_out=True)
        check_sequence(out[0], S[0], q[0], k[0], v[0], g[0], 1.0, s0[0], True)


STEPS = [(1, 1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 2, 64, 64), (5, 4, 2, 2, 4, 128, 128), (2, 3, 3, 3, 3, 48, 81), (40, 16, 16, 16, 16, 256, 512),
         (130, 4, 1, 4, 2, 80, 256), (2, 2, 2, 2, 2, 255, 20), (700, 1, 1, 1, 1, 33, 129), (1, 16, 16, 16, 16, 128, 128)]


@pytest.mark.parametrize("kind,out_kind", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("S,H,Hq,Hk,Hv,dk,dv", STEPS)
def test_step(kind, out_kind, S, H, Hq, Hk, Hv, dk, dv):
    q, k, v, g = inputs(S, H, Hq, Hk, Hv, 1, dk, dv, kind, S + dk, resets=0.1)
    gen = torch.Generator(DEV).manual_seed(8)
    pool = torch.randn(S + 2, H, dk, dv, device=DEV, generator=gen)
    order = np.random.default_rng(S).permutation(S + 2)[:S].astype(np.int32)
    if S > 2:
        order[1], order[2] = -1, S + 2
    before = pool.clone()
    out = rn().rn_linear_attention_step(q, k, v, g, pool, slots=torch.tensor(order, device=DEV), qk_scale=0.3,
                                        out_dtype=DT[out_kind])
    plain = before[:S].clone()
    out2 = rn().rn_linear_attention_step(q, k, v, g, plain, qk_scale=0.3, out_dtype=DT[out_kind])
    for s in list(range(min(S, 6))) + [S - 1]:
        args = (q[s], k[s], v[s], g[s], 0.3)
        check_sequence(out2[s], plain[s], *args, before[s])
        if 0 <= order[s] < S + 2:
            check_sequence(out[s], pool[order[s]], *args, before[order[s]])
        else:
            assert int(torch.count_nonzero(out[s])) == 0
    for i in set(range(S + 2)) - set(order.tolist()):
        assert torch.equal(pool[i], before[i])


def test_prompt_then_steps_is_one_sequence():
    """A prompt of 100 tokens and 20 steps on its state, against one prompt of 120 tokens."""
    B, H, N, d = 3, 4, 120, 64
    for kind in ("f32", "bf16"):
        q, k, v, g = inputs(B, H, H, H, H, N, d, d, kind, 16, True)
        cut = lambda t, a, b: t[:, :, a:b]  # noqa: E731
        first, S = rn().rn_linear_attention_chunked(*(cut(t, 0, 100) for t in (q, k, v, g)), state_out=True)
        outs = [first] + [rn().rn_linear_attention_step(*(cut(t, i, i + 1) for t in (q, k, v, g)), S) for i in range(100, N)]
        got = torch.cat(outs, 2)
        for b in range(B):
            check_sequence(got[b], S[b], q[b], k[b], v[b], g[b], 1.0, None, kind == "bf16")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_long_sequence_in_segments(kind):
    """A sequence long enough to be cut into segments: outputs and state against the oracle."""
    H, N, dk, dv = 2, 3000, 32, 64
    q, k, v, g = inputs(1, H, 1, 1, H, N, dk, dv, kind, 17, True, fade=16.0)
    assert rn().rn_linear_attention_workspace_bytes(q, k, v, g) > 0
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, state_out=True, qk_scale=0.2)
    check_sequence(out[0], S[0], q[0], k[0], v[0], g[0], 0.2, None, kind == "bf16")
    ws = torch.empty(rn().rn_linear_attention_workspace_bytes(q, k, v, g), dtype=torch.uint8, device=DEV).fill_(255)
    o2, S2 = rn().rn_linear_attention_chunked(q, k, v, g, state_out=True, qk_scale=0.2, workspace=ws)
    assert torch.equal(out, o2) and torch.equal(S, S2)                # the same bits, whatever the workspace held
    with pytest.raises(rn().RnError, match="RN_ERR_WORKSPACE"):
        rn().rn_linear_attention_chunked(q, k, v, g, workspace=ws[:256])


def test_offsets_past_32_bits():
    """A pool whose last state starts more than 2^32 bytes in, and token rows as far apart."""
    H, dk, dv = 16, 128, 256
    n = (1 << 32) // (4 * H * dk * dv) + 2
    pool = torch.zeros(n, H, dk, dv, device=DEV)
    q, k, v, g = inputs(1, H, H, H, H, 3, dk, dv, "bf16", 18)
    slots = torch.tensor([n - 1], dtype=torch.int32, device=DEV)
    out, _ = rn().rn_linear_attention_chunked(q, k, v, g, state_in=pool, state_out=pool, slots=slots)
    check_sequence(out[0], pool[n - 1], q[0], k[0], v[0], g[0], 1.0, None, True)
    assert int(torch.count_nonzero(pool[0])) == 0
    keep = pool[n - 1].clone()
    one = [t[:, :, :1] for t in (q, k, v, g)]
    out = rn().rn_linear_attention_step(*one, pool, slots=slots)
    check_sequence(out[0], pool[n - 1], *(t[0] for t in one), 1.0, keep)
    del pool
    wide = torch.zeros((1 << 31) + 4096, dtype=torch.bfloat16, device=DEV)      # two token rows 2^31 elements apart
    far = wide.as_strided((1, 2, 2, 64), (0, 64, 1 << 31, 1))
    q, k, v, g = inputs(1, 2, 2, 2, 2, 2, 64, 64, "bf16", 19)
    far.copy_(v)
    a, _ = rn().rn_linear_attention_chunked(q, k, far, g)
    b, _ = rn().rn_linear_attention_chunked(q, k, v, g)
    assert torch.equal(a, b)


@pytest.mark.parametrize("kind,generic", [("bf16", False), ("bf16", True), ("f32", False)])
def test_many_segments(kind, generic):
    """More segments than the scan holds in flight, of a padded batch with a short and an empty
    sequence beside the long one; the final state, and one without."""
    B, H, N, d = 3, 1, 9000, 16
    q, k, v, g = inputs(B, H, H, H, H, N, d, d, kind, 21, True, fade=16.0)
    s0 = torch.randn(B, H, d, d, device=DEV, generator=torch.Generator(DEV).manual_seed(9))
    lens = [9000, 5, 0]
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, lengths=ln, state_in=s0, state_out=True, force_generic=generic)
    drop, _ = rn().rn_linear_attention_chunked(q, k, v, g, lengths=ln, state_in=s0, force_generic=generic)
    assert torch.equal(out, drop) and torch.equal(S[2], s0[2])
    for b in range(2):
        n = lens[b]
        check_sequence(out[b, :, :n], S[b], q[b, :, :n], k[b, :, :n], v[b, :, :n], g[b, :, :n], 1.0, s0[b], kind == "bf16" and not generic)


@pytest.mark.parametrize("N", [100, 2000])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 8), (0, 3), (1, 7), (3, 0), (8, 24)])
def test_views_of_a_projection(N, off, pad):
    """q, k, v as slices of one bf16 buffer at odd places and strides, out into a buffer of its
    own with gaps, which keep their bits; 16-byte rows or not, the numbers hold."""
    H, dk, dv = 2, 32, 40
    cols = H * (2 * dk + dv) + pad
    g_ = torch.Generator().manual_seed(22 + off + pad)
    buf = torch.randn(1, N, off + cols, generator=g_).bfloat16().to(DEV)
    dec = torch.nn.functional.logsigmoid(torch.randn(1, H, N, generator=g_) + 2).to(DEV) / 4
    cut = lambda c0, d: buf[..., off + c0:off + c0 + H * d].unflatten(-1, (H, d)).transpose(1, 2)  # noqa: E731
    q, k, v = cut(0, dk), cut(H * dk, dk), cut(2 * H * dk, dv)
    wide = torch.full((1, N, off + H * dv + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    out = wide[..., off:off + H * dv].unflatten(-1, (H, dv)).transpose(1, 2)
    ws = torch.empty(rn().rn_linear_attention_workspace_bytes(q, k, v, dec, out=out) or 16, dtype=torch.uint8, device=DEV)
    _, S = rn().rn_linear_attention_chunked(q, k, v, dec, out=out, state_out=True, workspace=ws)
    check_sequence(out[0], S[0], q[0], k[0], v[0], dec[0], 1.0, None, True)
    assert (wide[..., :off] == 7.0).all() and (wide[..., off + H * dv:] == 7.0).all()


@pytest.mark.parametrize("scale", [-0.7, 0.0, 1e-30, 1e4])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scales(kind, scale):
    q, k, v, g = inputs(1, 2, 2, 2, 2, 150, 64, 64, kind, 23)
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=scale, state_out=True)
    o, _ = K.linear_attention(q[0], k[0], v[0], g[0], scale)
    if scale == 0.0:
        assert int(torch.count_nonzero(out)) == 0
    else:
        check_sequence(out[0], S[0], q[0], k[0], v[0], g[0], scale, None, kind == "bf16")
    ref, R = rn().rn_linear_attention_chunked(q, k, v, g, state_out=True)
    assert torch.equal(S, R)                               # the scale never enters the state


def test_two_graphs_on_one_workspace():
    """Two captured calls that share a workspace, replayed in turn, against eager calls."""
    sets = [inputs(1, 2, 2, 2, 2, 2000, 64, 64, "bf16", s) for s in (24, 25)]
    n = rn().rn_linear_attention_workspace_bytes(*sets[0])
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    run = lambda t: rn().rn_linear_attention_chunked(*t, state_out=True, workspace=ws)  # noqa: E731
    want = [tuple(x.clone() for x in run(t)) for t in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for t in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(run(t))
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 1):
        ws.fill_(255)
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[turn], want[turn]))


def test_refusals():
    q, k, v, g = inputs(2, 4, 4, 2, 4, 8, 16, 16, "f32", 20)
    f, st = rn().rn_linear_attention_chunked, rn().rn_linear_attention_step
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    S = torch.zeros(2, 4, 16, 16, device=DEV)
    for args, kw in (((q, k[:1], v, g), {}), ((q, k, v[:, :, :7], g), {}), ((q, k, v, g[:, :, :7]), {}), ((q, k, v, g.double()), {}),
                     ((q[0], k[0], v[0], g[0]), {}), ((q, k, v, g), dict(lengths=i32(1))), ((q, k, v, g), dict(lengths=torch.tensor([1, 2], device=DEV))),
                     ((q, k, v, g), dict(cu_seqlens=i32(0, 8))), ((q, k, v, g), dict(state_in=S[:1])), ((q, k, v, g), dict(state_in=S.bfloat16())),
                     ((q, k, v, g), dict(state_in=S.transpose(2, 3))), ((q, k, v, g), dict(out=torch.zeros(2, 4, 8, 17, device=DEV))),
                     ((q, k, v, g), dict(max_len=9)), ((q, k, v, g), dict(max_len=0)), ((q, k, v, g), dict(slots=i32(0, 1), state_out=True)),
                     ((q, k, v, g), dict(slots=i32(0), state_in=S)), ((q, k, v, g), dict(slots=i32(0, 1), state_in=S, state_out=S[:1])),
                     ((q, k, v, g.cpu()), {}), ((q.transpose(2, 3), k, v, g), {}), ((q, k, v, g), dict(workspace=S))):
        with pytest.raises(ValueError):
            f(*args, **kw)
    with pytest.raises(TypeError):
        f(q, k, v.bfloat16(), g)
    with pytest.raises(TypeError):
        f(q.half(), k.half(), v.half(), g)
    with pytest.raises(rn().RnError):
        f(q[:, :3], k, v, g)                               # 3 heads do not divide 4
    with pytest.raises(rn().RnError):
        f(q, k, v, g, out=torch.zeros(2, 1, 8, 16, device=DEV).expand(2, 4, 8, 16))
    with pytest.raises(ValueError):
        st(q, k, v, g, S)                                  # 8 tokens
    one = [t[:, :, :1] for t in (q, k, v, g)]
    with pytest.raises(ValueError):
        st(*one, S[:1])
    with pytest.raises(ValueError):
        st(*one, S, slots=i32(0))


@pytest.mark.parametrize("kind,dk,dv", [("f32", 33, 24), ("bf16", 64, 64), ("bf16", 256, 96)])
@pytest.mark.parametrize("longest", [300, 2100])
def test_many_packed_sequences_without_a_bound(kind, dk, dv, longest):
    """Forty sequences, most of one segment or none, one longer, with no nearer bound on their
    lengths than the rows of all: outputs, states (in place, in a pool, some without a slot), the
    sequences without tokens and the rows behind the last; then an out that is given, and a bound
    that cuts the longest sequence."""
    gen = np.random.default_rng(21)
    S, H = 40, 2
    lens = gen.integers(0, 60, S)
    lens[[0, 7, 39]] = 0
    lens[11] = longest
    T = int(lens.sum()) + 70
    q, k, v, g = inputs(1, H, 1, H, 2, T, dk, dv, kind, 22, True)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    e = int(lens.sum())
    for t in (q, k, v, g):
        t[:, :, e:] = float("nan")
    pool = torch.randn(S + 2, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(8))
    before = pool.clone()
    order = gen.permutation(S + 2)[:S].astype(np.int32)
    order[[3, 11 if longest < 1000 else 12]] = -1
    slots = torch.tensor(order, device=DEV)
    out, _ = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, state_in=pool, state_out=pool, slots=slots)
    assert (out[:, :, e:] == 0.0).all()
    for s in range(S):
        a, b, slot = int(cu[s]), int(cu[s + 1]), int(order[s])
        if b > a:
            check_sequence(out[0, :, a:b], pool[slot] if slot >= 0 else None, q[0, :, a:b], k[0, :, a:b], v[0, :, a:b],
                           g[0, :, a:b], 1.0, before[slot] if slot >= 0 else None, uses_mfma(kind, DT[kind], dk, dv, False))
        elif slot >= 0:
            assert torch.equal(pool[slot], before[slot])
    for i in set(range(S + 2)) - set(order.tolist()):
        assert torch.equal(pool[i], before[i])
    mine = torch.full_like(out, 7.0)
    _, new = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, state_out=True, out=mine)
    assert (mine[:, :, e:] == 7.0).all() and int(torch.count_nonzero(new[7])) == 0
    a = int(cu[11])
    stop = longest - 100
    cut, _ = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, max_len=stop, state_out=True)
    assert (cut[:, :, a + stop:a + longest] == 0.0).all() and (cut[:, :, e:] == 0.0).all()
    check_sequence(cut[0, :, a:a + stop], None, q[0, :, a:a + stop], k[0, :, a:a + stop], v[0, :, a:a + stop],
                   g[0, :, a:a + stop], 1.0, None, uses_mfma(kind, DT[kind], dk, dv, False))


def test_flat_grid_without_tokens_and_with_disordered_bounds():
    """Every sequence without tokens; entries outside the tensors and out of order: nothing is
    written outside."""
    H, dk, dv, T, S = 2, 64, 64, 2000, 50
    q, k, v, g = inputs(1, H, H, H, H, T, dk, dv, "bf16", 23, True)
    none = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    s0 = torch.randn(S, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(9))
    out, new = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=none, state_in=s0, state_out=True)
    assert int(torch.count_nonzero(out)) == 0 and torch.equal(new, s0)
    guard = torch.full((T + 200, H, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    o = guard[100:100 + T].transpose(0, 1)[None]
    bad = np.random.default_rng(24).integers(-3000, 5000, S + 1).astype(np.int32)
    for generic in (True, False):
        rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=torch.tensor(bad, device=DEV), out=o, state_out=True,
                                         force_generic=generic)
    torch.cuda.synchronize()
    assert (guard[:100] == 7.0).all() and (guard[100 + T:] == 7.0).all()


@pytest.mark.parametrize("dk,dv,N,scale", [(64, 64, 200, 0.125), (16, 40, 700, -1.5), (128, 128, 900, 1.0), (256, 96, 130, 0.0625),
                                           (256, 512, 150, 0.0625), (256, 512, 900, 1.0), (192, 256, 850, 0.3)])
def test_bf16_prompts_are_rounded_once(dk, dv, N, scale):
    """A bf16 output is the float32 result rounded once (H16 of it). Scores, the state's copy that
    queries read, and the tokens' shares of the state in a pass that only gives outputs are held in
    two bf16 parts: what is left of a value after two roundings is at most H16^2 = 2^-16 of it. A
    score or a state value meets one such loss on its own side and one in the tokens behind it: 2
    H16^2 M beside the float32 bound c M. (1 and 3 segments at each width of the state.)"""
    H = 2
    q, k, v, g = inputs(1, H, H, H, H, N, dk, dv, "bf16", 26 + dk, True, fade=16.0, resets=0.002)
    s0 = torch.randn(1, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(10))
    for want in (True, False):
        out, _ = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=scale, state_in=s0, state_out=want)
        o, _ = K.linear_attention(q[0], k[0], v[0], g[0], scale, s0[0])
        mo, _ = K.linear_attention(q[0].abs(), k[0].abs(), v[0].abs(), g[0], abs(scale), s0[0].abs())
        c = (3 * reach(g[0]) + dk + 64) * U
        tol = (c + 2 * H16 * H16) * mo * (1 + 2 * H16) + H16 * np.abs(o) + 1e-30
        off = np.abs(np64(out[0]) - o)
        assert (off <= tol).all(), f"{(off / tol).max()} of the tolerance at {np.unravel_index((off / tol).argmax(), off.shape)}"


@pytest.mark.parametrize("dk,dv,N", [(64, 64, 70), (128, 128, 900), (256, 512, 130), (256, 64, 70)])
def test_infinite_states_stay_infinite(dk, dv, N):
    """An infinity in the starting state reaches its column of every output, as an infinity of the
    sign that the query gives it, and no other column."""
    q, k, v, g = inputs(1, 2, 2, 2, 2, N, dk, dv, "bf16", 27, True, fade=16.0)
    s0 = torch.randn(1, 2, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(11))
    q[..., 5] = torch.where(q[..., 5] == 0, 1.0, q[..., 5])
    clean, _ = rn().rn_linear_attention_chunked(q, k, v, g, state_in=s0)
    s0[0, 1, 5, 7] = float("inf")
    base, _ = rn().rn_linear_attention_chunked(q, k, v, g, state_in=s0)
    sign = torch.sign(q[0, 1, :, 5].float())
    assert torch.equal(base[0, 1, :, 7].float(), sign * float("inf"))
    rest = [c for c in range(dv) if c != 7]
    assert torch.equal(base[0, 0], clean[0, 0]) and torch.equal(base[0, 1][:, rest], clean[0, 1][:, rest])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (256, 512)])
def test_decays_behind_many_resets(dk, dv):
    """Fifty zero decays, then mild ones, in one chunk: the sums of log decays are far from zero where
    the differences that count are small. Tolerance as for outputs that are rounded once."""
    H, N, scale = 2, 128, 0.37
    q, k, v, g = inputs(1, H, H, H, H, N, dk, dv, "bf16", 28 + dk, True, fade=16.0)
    g[:, :, 3:53] = -float("inf")
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=scale, state_out=True)
    o, So = K.linear_attention(q[0], k[0], v[0], g[0], scale)
    mo, mS = K.linear_attention(q[0].abs(), k[0].abs(), v[0].abs(), g[0], scale)
    c = (3 * reach(g[0]) + dk + 64) * U
    off, tol = np.abs(np64(out[0]) - o), (c + 2 * H16 * H16) * mo * (1 + 2 * H16) + H16 * np.abs(o) + 1e-30
    assert (off <= tol).all(), f"{(off / tol).max()} of the tolerance at {np.unravel_index((off / tol).argmax(), off.shape)}"
    off, tol = np.abs(np64(S[0]) - So), c * mS + 1e-30
    assert (off <= tol).all(), f"state: {(off / tol).max()} of the tolerance"


@pytest.mark.parametrize("kind,dk,dv", [("bf16", 64, 64), ("bf16", 256, 512), ("f32", 64, 64)])
def test_a_reset_clears_the_state_at_any_scale(kind, dk, dv):
    """Nothing of a large state is left behind a zero decay, whatever the scale."""
    q, k, v, g = inputs(1, 2, 2, 2, 2, 70, dk, dv, kind, 29)
    k.zero_()
    g[:, :, 1] = -float("inf")
    s0 = torch.full((1, 2, dk, dv), 1e30, device=DEV)
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, qk_scale=1e25, state_in=s0, state_out=True)
    assert int(torch.count_nonzero(out[:, :, 1:])) == 0 and int(torch.count_nonzero(S)) == 0


@pytest.mark.parametrize("kind,dk,dv,L", [("f32", 33, 24, 64), ("bf16", 64, 64, 256), ("bf16", 256, 96, 256)])
def test_flat_grid_with_many_sequences_of_several_segments(kind, dk, dv, L):
    """Sequences just above, at and below whole numbers of segments (of L tokens here), short ones
    between: every state and output, into a workspace of just the bytes asked for, and nothing
    behind it."""
    H = 2
    lens = [L + 1, 1, L + 1, 2 * L + 1, 0, L, L + 1, 3, 2 * L, L + 2, L - 1, 3 * L + 1, 0, L + 1, L + 1, 5]
    S, T = len(lens), sum(lens)
    q, k, v, g = inputs(1, H, H, 1, H, T, dk, dv, kind, 30, True, fade=16.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    s0 = torch.randn(S, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(12))
    need = rn().rn_linear_attention_workspace_bytes(q, k, v, g, cu_seqlens=cu)
    assert need > 0
    guard = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    out, new = rn().rn_linear_attention_chunked(q, k, v, g, cu_seqlens=cu, state_in=s0, state_out=True, workspace=guard[:need])
    assert (guard[need:] == 77).all()
    for s in range(S):
        a, b = int(cu[s]), int(cu[s + 1])
        if b > a:
            check_sequence(out[0, :, a:b], new[s], q[0, :, a:b], k[0, :, a:b], v[0, :, a:b], g[0, :, a:b], 1.0, s0[s],
                           uses_mfma(kind, DT[kind], dk, dv, False))
        else:
            assert torch.equal(new[s], s0[s])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("S,H,dk,dv", [(130, 4, 128, 192), (33, 16, 128, 320), (64, 8, 64, 384), (520, 1, 256, 448), (520, 1, 192, 384)])
def test_step_in_several_whole_slices(kind, S, H, dk, dv):
    """Enough states for the kernel whose threads all have columns and rows, and values of two to seven
    of its widths of columns."""
    q, k, v, g = inputs(S, H, H, 1, H, 1, dk, dv, kind, S + dv, resets=0.1)
    state = torch.randn(S, H, dk, dv, device=DEV, generator=torch.Generator(DEV).manual_seed(13))
    before = state.clone()
    out = rn().rn_linear_attention_step(q, k, v, g, state, qk_scale=0.3)
    for s in (0, 1, S // 2, S - 1):
        check_sequence(out[s], state[s], q[s], k[s], v[s], g[s], 0.3, before[s])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dk,dv,N", [(64, 64, 200), (128, 64, 900), (256, 96, 200), (256, 512, 900)])
def test_columns_beside_a_nonfinite_value_keep_their_precision(bad, dk, dv, N):
    """Chunks whose values are not all finite are added up another way: the other columns' outputs are
    rounded once there too, at every width of the state, in one pass and over segments."""
    H = 2
    q, k, v, g = inputs(1, H, H, H, H, N, dk, dv, "bf16", 31 + dk, True, fade=16.0)
    rest = [c for c in range(dv) if c != 5]
    v[0, 1, 100, 5] = bad
    out, S = rn().rn_linear_attention_chunked(q, k, v, g, state_out=True, qk_scale=0.1)
    o, So = K.linear_attention(q[0], k[0], v[0], g[0], 0.1)
    assert np.array_equal(np.isfinite(np64(out[0])), np.isfinite(o)) and np.array_equal(np.isfinite(np64(S[0])), np.isfinite(So))
    assert not np.isfinite(o[1, 100:, 5]).any() and np.isfinite(o[1, :100]).all()
    o, So = o[..., rest], So[..., rest]
    mo, mS = K.linear_attention(q[0].abs(), k[0].abs(), v[0][..., rest].abs(), g[0], 0.1)
    c = (3 * reach(g[0]) + dk + 64) * U
    off, tol = np.abs(np64(out[0])[..., rest] - o), (c + 2 * H16 * H16) * mo * (1 + 2 * H16) + H16 * np.abs(o) + 1e-30
    assert (off <= tol).all(), f"{(off / tol).max()} of the tolerance at {np.unravel_index((off / tol).argmax(), off.shape)}"
    assert (np.abs(np64(S[0])[..., rest] - So) <= c * mS + 1e-30).all()
