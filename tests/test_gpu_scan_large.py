"""The short convolution and the selective scan at sizes that take their kernels' other ways: pieces of several
tiles, steps of two sequences a thread, blocks that walk along pieces, and more pieces than a grid's axis has.
Tolerances as in the files of the small sizes, where not said otherwise."""
import numpy as np
import pytest
import torch

from oracle import scan as O
from tests import test_gpu_short_conv as conv
from tests.test_gpu_selective_scan import HALF, U, Batch, bounds, f64, rn
from tests.test_gpu_selective_scan_backward import batch, check, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def tokens_a_piece(b):
    """Tokens a piece of the gradients' call, from its workspace: two states and three sums a piece and channel,
    and two rows of n a token and block along the channels."""
    need = rn().rn_selective_scan_backward_workspace_bytes(b.x, b.A, b.B, cu_seqlens=b.kw.get("cu_seqlens"))
    S, (rows, N) = len(b.lens), b.x.shape[:2]
    blocks = b.G * -(-(b.D // b.G) // 64)
    pieces = (need // 4 - rows * N * blocks * 2 * b.n) // (b.D * (2 * b.n + 3))
    return next(k for k in (32, 16, 8, 4, 2) if pieces == (N // k + S + 1 if b.packed else S * -(-N // k)))


SHORT = [70, 0, 61, 9]
SEVERAL = [(SHORT, 512, 1, 512, 32), (SHORT, 512, 4, 512, 32), (SHORT, 512, 5, 512, 32), (SHORT, 512, 12, 512, 32), (SHORT, 512, 16, 512, 32),
           (SHORT, 256, 16, 256, 16), (SHORT, 256, 8, 256, 16), (SHORT, 128, 24, 128, 32), (SHORT, 64, 20, 64, 16), (SHORT, 64, 33, 64, 16),
           (SHORT, 32, 40, 32, 8), (SHORT, 64, 64, 64, 16)]


@pytest.mark.parametrize("lens,D,n,G,tokens", SEVERAL)
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_pieces_of_several_tiles(lens, D, n, G, tokens, kind, packed):
    for k, (kw, softplus) in enumerate([(dict(), True), (dict(view=1, start=False), True), (dict(bias=False, gate=False), False)]):
        b = batch(D * 3 + n + k, lens, D, n, G, kind, packed, **kw)
        assert tokens_a_piece(b) >= tokens and (not packed or tokens_a_piece(b) == tokens)
        if not softplus:
            b.dt = b.dt.abs() * 0.1            # steps as they are
        check(b, run(b, softplus, dstate_out=b.dstate, want_dstate_in=True), softplus, kind, b.dstate)


@pytest.mark.parametrize("D,n,G", [(8192, 4, 128), (4160, 12, 64), (2112, 24, 33)])
def test_gradients_of_pieces_of_several_tiles_and_waves_of_many_channels(D, n, G):
    b = batch(n, [300, 211], D, n, G, torch.float32, True)
    assert tokens_a_piece(b) == 32
    check(b, run(b, dstate_out=b.dstate, want_dstate_in=True), True, torch.float32, b.dstate)


@pytest.mark.parametrize("D,n,G,S", [(4096, 16, 1, 65), (4096, 5, 2, 33), (8192, 4, 8, 129), (1000, 64, 1, 263)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_many_single_tokens(D, n, G, S, kind):
    """Two sequences a thread: an odd number of them, skipped ones beside others, against the oracle and bit by bit
    against a few sequences at a time."""
    b = Batch(D + n, [1] * S, D, n, G, kind, False, pad=0)
    g = torch.Generator().manual_seed(S)
    slots = torch.randperm(S + 3, generator=g)[:S].int()
    skipped = [0, 3, 4, 5, 8, 11, S - 2]
    slots[skipped] = torch.tensor([-1, S + 3, -5, 1 << 30, S + 900, -1, -1], dtype=torch.int32)
    slots = slots.to(DEV)
    pool = torch.randn(S + 3, D, n, generator=g).to(DEV)
    before, part = pool.clone(), pool.clone()

    def step(pool, a, e):
        return rn().rn_selective_scan_step(b.x[a:e], b.dt[a:e], b.A, b.B[a:e], b.C[a:e], pool, b.skip, dt_bias=b.bias, z=b.z[a:e],
                                           slots=slots[a:e])
    out = step(pool, 0, S)
    few = torch.cat([step(part, a, min(a + 3, S)) for a in range(0, S, 3)])
    assert torch.equal(out, few) and torch.equal(pool, part)
    used = {int(slots[s]): s for s in range(S) if s not in skipped}
    for i in range(S + 3):
        if i not in used:
            assert torch.equal(pool[i], before[i])
    for i, s in list(used.items())[::7] + [(int(slots[S - 1]), S - 1)]:
        p = {**b.sequence(s, (s, slice(0, 1))), "state": f64(before[i])}
        want, h = O.selective_scan(**p)
        yb, hb = bounds(p, True)
        assert (np.abs(f64(out[s]) - want) <= yb + HALF[kind] * np.abs(want) + 1e-37).all()
        assert (np.abs(f64(pool[i]) - h) <= hb + 1e-37).all()
    assert (out[skipped] == 0).all()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_convolution_gradients_of_blocks_that_walk_along_pieces(packed, kind):
    """More than 128 pieces of 32 tokens: a thread sums runs of 8 tokens of several pieces, a block its 4 runs, and 4
    and 32 sums of the 128 rows of blocks follow."""
    D, K = 256, 4
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 40, 400)] if packed else [2500, 2497]
    b = conv.Batch(5, lens, D, K, kind, packed)
    rows = b.x.shape[1]
    pieces = rows // 32 + len(lens) + 1 if packed else len(lens) * -(-rows // 32)
    assert pieces > 128
    roundings = -(-pieces // 128) * 8 + 4 + 4 + 32
    got = rn().rn_short_conv_backward(b.dy, b.x, b.w, b.b, silu=True, state_in=b.state, dstate_out=b.dstate, want_dstate_in=True, **b.kw)
    assert (b.rest(got["dx"]) == 0).all()
    w = f64(b.w)
    dw, db, bw, bb = np.zeros_like(w), np.zeros(D), np.zeros_like(w), np.zeros(D)
    for i, at, _ in b.spans():
        s, x, dy = f64(b.state[i]), f64(b.x[at]), f64(b.dy[at])
        wx, ww, wb, ws = O.short_conv_backward(dy, x, w, f64(b.b), True, s, f64(b.dstate[i]))
        u, _ = O.short_conv(x, w, f64(b.b), False, s)
        size = np.abs(dy) * 1.1
        per = np.abs(dy) * ((np.abs(u) * 2 + 16) * U + 0.6 * (K + 1) * U * conv.sizes(x, w, f64(b.b), s)) + (K + 2) * U * size
        dxo, dwo, dbo, dso = O.short_conv_backward(per, np.abs(x), np.abs(w), None, False, np.abs(s), U * np.abs(f64(b.dstate[i])))
        assert (np.abs(f64(got["dx"][at]) - wx) <= dxo + HALF[kind] * np.abs(wx) + 1e-37).all(), i
        assert (np.abs(f64(got["dstate_in"][i]) - ws) <= dso + U * np.abs(ws) + 1e-37).all(), i
        _, dws, dbs, _ = O.short_conv_backward(size, np.abs(x), np.abs(w), None, False, np.abs(s))
        dw += ww
        db += wb
        bw += dwo + roundings * U * dws
        bb += dbo + roundings * U * dbs
    assert (np.abs(f64(got["dweight"]) - dw) <= bw + 1e-37).all() and (np.abs(f64(got["dbias"]) - db) <= bb + 1e-37).all()


def test_more_pieces_than_a_grids_axis():
    """65534 packed sequences of 0 to 3 tokens against the same ones padded: the same bits a token, and sums of
    positive terms within the roundings of 32 interleaved sums of the pieces (at most 4000 each time)."""
    S, D, n = 65534, 8, 4
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 4, (S,), generator=g)
    live = (torch.arange(3)[None] < lens[:, None]).to(DEV)
    cu = torch.cat([torch.zeros(1), lens.cumsum(0)]).int().to(DEV)
    lens = lens.int().to(DEV)
    r = lambda *s: (torch.rand(*s, generator=g) + 0.1).to(DEV)  # noqa: E731
    pack = lambda t: t[live][None].contiguous()  # noqa: E731
    x, dt, dy, w, bias = r(S, 3, D), r(S, 3, D), r(S, 3, D), r(D, 4), r(D)
    pad, packed = dict(lengths=lens), dict(cu_seqlens=cu, max_len=3)
    state = r(S, 3, D)
    a, b = (rn().rn_short_conv(t, w, bias, state_in=state, state_out=True, **kw) for t, kw in ((x, pad), (pack(x), packed)))
    assert torch.equal(pack(a[0]), b[0]) and torch.equal(a[1], b[1])
    a, b = (rn().rn_short_conv_backward(d, t, w, bias, state_in=state, want_dstate_in=True, **kw)
            for d, t, kw in ((dy, x, pad), (pack(dy), pack(x), packed)))

    def same(tokens):
        for k in a:
            if k in tokens:
                assert torch.equal(pack(tokens[k](a[k])), tokens[k](b[k])), k
            elif k == "dstate_in":
                assert torch.equal(a[k], b[k])
            else:
                assert (a[k] - b[k]).abs().max() <= 8000 * U * a[k].abs().max() and a[k].min() != 0, k
    same({"dx": lambda t: t})
    A, B, C, state = -r(D, n), r(S, 1, 3, n), r(S, 1, 3, n), r(S, D, n)
    heads = lambda t: pack(t[:, 0])[:, None]  # noqa: E731
    a, b = (rn().rn_selective_scan_chunked(x_, dt_, A, B_, C_, w[:, 0].contiguous(), state_in=state, state_out=True, **kw)
            for x_, dt_, B_, C_, kw in ((x, dt, B, C, pad), (pack(x), pack(dt), heads(B), heads(C), packed)))
    assert torch.equal(pack(a[0]), b[0]) and torch.equal(a[1], b[1])
    a, b = (rn().rn_selective_scan_backward(d_, x_, dt_, A, B_, C_, state_in=state, want_dstate_in=True, **kw)
            for d_, x_, dt_, B_, C_, kw in ((dy, x, dt, B, C, pad), (pack(dy), pack(x), pack(dt), heads(B), heads(C), packed)))
    one = lambda t: t[:, 0]  # noqa: E731
    same({"dx": lambda t: t, "ddt": lambda t: t, "dB": one, "dC": one})
