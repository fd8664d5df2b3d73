"""Host-side checks of the operators around retention (no GPU needed): invalid arguments are
rejected before any HIP call. Pointers passed here are never dereferenced."""
import ctypes
import math

import numpy as np
import pytest
import torch

import linear_recurrent_sequence_rn_amd as rn

FAKE = 0x10000
L = rn.lib
INV, UNS, WS = rn.RN_ERR_INVALID_ARG, rn.RN_ERR_UNSUPPORTED, rn.RN_ERR_WORKSPACE


def fill(cls, base, kw):
    d = cls()
    for name, v in {**base, **kw}.items():
        if isinstance(v, tuple):
            v = (ctypes.c_int64 * 3)(*v)
        setattr(d, name, v)
    return d


def norm(**kw):
    return fill(rn.RnNormDesc, dict(rows=4, d=64, in_dtype=1, out_dtype=1, eps=1e-5, x_stride=64, res_stride=64,
                                    sum_stride=64, out_stride=64), kw)


def norm_forward(d, x=FAKE, r=None, s=None, out=2 * FAKE):
    return L.rn_layernorm_forward(ctypes.byref(d), x, r, None, None, s, out, None)


def norm_backward(d, dout=FAKE, x=FAKE, dx=2 * FAKE, dw=FAKE, ws=FAKE, n=1 << 40):
    return L.rn_layernorm_backward(ctypes.byref(d), dout, x, None, None, dx, dw, None, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(d=0), INV), (dict(d=16385), UNS), (dict(rows=(1 << 40) + 1), UNS),
    (dict(in_dtype=2), INV), (dict(out_dtype=-1), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(eps=math.inf), INV), (dict(x_stride=-64), INV), (dict(res_stride=(1 << 40) + 1), INV),
    (dict(out_stride=63), INV), (dict(sum_stride=10), INV)])
def test_norm_descriptors(kw, code):
    d = norm(**kw)
    out_only = "out_stride" in kw and kw["out_stride"] > 0
    assert norm_forward(d, s=3 * FAKE) == code and L.rn_last_error() != b""
    assert out_only or norm_backward(d) == code
    if not ({"out_stride", "sum_stride"} & set(kw)):
        assert L.rn_layernorm_backward_workspace_bytes(ctypes.byref(d)) == 0


def test_norm_pointers_and_workspace():
    d = norm()
    assert L.rn_layernorm_forward(None, FAKE, None, None, None, None, FAKE, None) == INV
    assert norm_forward(d, x=None) == INV and norm_forward(d, out=None) == INV
    assert norm_forward(d, x=FAKE + 1) == INV                       # bf16 on an odd address
    assert norm_forward(d, s=2 * FAKE) == INV                       # out and sum_out the same
    assert norm_forward(norm(out_dtype=0), x=FAKE, out=FAKE) == INV  # in place with other types
    assert norm_forward(norm(out_stride=128), x=FAKE, out=FAKE) == INV
    assert norm_backward(d, dx=None) == INV and norm_backward(d, dout=None) == INV
    assert norm_backward(d, dx=FAKE, dout=FAKE, x=5 * FAKE, ws=None) == WS
    need = L.rn_layernorm_backward_workspace_bytes(ctypes.byref(d))
    assert need > 0 and norm_backward(d, n=need - 1) == WS
    assert norm_backward(d, ws=FAKE + 16) == INV
    assert norm_backward(norm(out_dtype=0), dout=FAKE, dx=FAKE) == INV


TH = np.ones(128)


def rot(**kw):
    s = (4096, 512, 128)
    return fill(rn.RnRotaryDesc, dict(B=1, N=4, H_q=8, H_k=8, d=128, rot=128, dtype=1, flags=0, pos0=0, magnitude=1.0,
                                      theta=TH.ctypes.data, q_stride=s, k_stride=s, q_out_stride=s, k_out_stride=s), kw)


def rotary(d, pos=None, q=FAKE, k=2 * FAKE, qo=3 * FAKE, ko=4 * FAKE):
    return L.rn_rotary(ctypes.byref(d), pos, q, k, qo, ko, None)


BAD_TH = np.full(128, np.nan)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INV), (dict(N=0), INV), (dict(H_q=0), INV), (dict(H_k=-1), INV), (dict(d=1), INV),
    (dict(rot=0), INV), (dict(rot=127), INV), (dict(rot=130), INV), (dict(d=513), UNS),
    (dict(d=512, rot=258), UNS), (dict(H_q=65530, H_k=6), UNS), (dict(B=1 << 16, N=1 << 15), UNS),
    (dict(dtype=2), INV), (dict(flags=8), INV), (dict(pos0=-1), INV), (dict(pos0=(1 << 40) + 1), INV),
    (dict(magnitude=math.inf), INV), (dict(theta=None), INV), (dict(theta=BAD_TH.ctypes.data), INV),
    (dict(flags=4), INV), (dict(q_stride=(-1, 512, 128)), INV), (dict(q_out_stride=(4096, 0, 128)), INV),
    (dict(k_out_stride=(4096, 512, 127)), INV), (dict(q_out_stride=(0, 128, 512)), INV)])
def test_rotary_descriptors(kw, code):
    if kw.get("q_out_stride", (1,))[0] == 0:
        kw = dict(kw, B=2)
    assert rotary(rot(**kw)) == code and L.rn_last_error() != b""


def test_rotary_pointers():
    assert L.rn_rotary(None, None, FAKE, FAKE, FAKE, FAKE, None) == INV
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=FAKE + 1), dict(ko=4 * FAKE + 1),
               dict(pos=FAKE + 4), dict(qo=4 * FAKE)):
        assert rotary(rot(), **kw) == INV, kw
    assert rotary(rot(q_out_stride=(8192, 1024, 256)), qo=FAKE) == INV   # in place, other strides


def test_rotary_frequencies():
    t, m = rn.rn_rotary_frequencies(64)
    j = np.arange(32)
    assert m == 1.0 and np.abs(t / 10000.0 ** (-j / 32) - 1).max() < 1e-14
    t2, _ = rn.rn_rotary_frequencies(64, kind="linear", factor=4)
    assert np.abs(t2 * 4 / t - 1).max() < 1e-14
    t3, m3 = rn.rn_rotary_frequencies(64, kind="base", factor=4)
    assert m3 == 1.0 and t3[0] == 1.0 and abs(t3[-1] * 4 / t[-1] - 1) < 1e-12
    t4, m4 = rn.rn_rotary_frequencies(64, kind="by_parts", factor=8, length=4096, slow=1, fast=32)
    turns = 4096 * t / (2 * np.pi)
    assert abs(m4 - (0.1 * math.log(8) + 1)) < 1e-6
    assert np.array_equal(t4[turns >= 32], t[turns >= 32]) and (turns >= 32).any()
    assert np.abs(t4[turns <= 1] * 8 / t[turns <= 1] - 1).max() < 1e-14 and (turns <= 1).any()
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert np.abs(t4[mid] / (t[mid] * (keep + (1 - keep) / 8)) - 1).max() < 1e-13 and mid.any()
    for bad in (dict(rot=3), dict(rot=0), dict(rot=258), dict(rot=64, base=1.0), dict(rot=64, base=math.inf),
                dict(rot=64, kind="linear", factor=0.5), dict(rot=2, kind="base", factor=2),
                dict(rot=64, kind="by_parts", factor=2, slow=3, fast=3),
                dict(rot=64, kind="by_parts", factor=2, length=0), dict(rot=64, kind="linear", factor=math.nan)):
        with pytest.raises(rn.RnError):
            rn.rn_rotary_frequencies(**bad)
    with pytest.raises(ValueError):
        rn.rn_rotary_frequencies(64, kind="stretched")
    assert L.rn_rotary_frequencies(64, 1e4, 7, 1.0, 1.0, 0.0, 1.0, t.ctypes.data, t.ctypes.data) == INV
    assert L.rn_rotary_frequencies(64, 1e4, 0, 1.0, 1.0, 0.0, 1.0, None, None) == INV


def lin(**kw):
    s = (1 << 20, 1 << 14, 64)
    return fill(rn.RnLinearDesc, dict(S=2, N=100, H=8, H_q=8, H_k=8, H_v=8, d_k=64, d_v=64, in_dtype=1, out_dtype=1,
                                      flags=0, qk_scale=1.0, T=0, n_slots=0, q_stride=s, k_stride=s, v_stride=s,
                                      g_stride=(800, 100, 1), out_stride=s), kw)


def chunked(d, cu=None, lens=None, slots=None, q=FAKE, g=FAKE, s0=None, s1=None, out=FAKE, ws=FAKE, n=1 << 40):
    return L.rn_linear_attention_chunked(ctypes.byref(d), cu, lens, slots, q, FAKE, FAKE, g, s0, s1, out, ws, n, None)


def step(d, slots=None, state=FAKE, q=FAKE, out=FAKE):
    return L.rn_linear_attention_step(ctypes.byref(d), slots, q, FAKE, FAKE, FAKE, state, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=0), INV), (dict(H=0), INV), (dict(H_q=0), INV), (dict(H_k=3), INV), (dict(H_v=16), INV), (dict(d_k=0), INV),
    (dict(d_k=257), UNS), (dict(d_v=513), UNS), (dict(S=65535), UNS), (dict(H=65536, H_q=1, H_k=1, H_v=1), UNS),
    (dict(in_dtype=2), INV), (dict(out_dtype=9), INV), (dict(flags=2), INV), (dict(qk_scale=math.nan), INV),
    (dict(T=-1), INV), (dict(T=1 << 31), INV), (dict(q_stride=(0, -1, 1)), INV),
    (dict(out_stride=(1 << 20, 1 << 14, 63)), INV), (dict(out_stride=(1 << 20, 64, 64)), INV)])
def test_linear_descriptors(kw, code):
    assert chunked(lin(**kw)) == code and L.rn_last_error() != b""
    assert L.rn_linear_attention_workspace_bytes(ctypes.byref(lin(**kw))) == 0
    if "out_stride" not in kw:                          # the step has one token: any token stride
        assert step(lin(**{"N": 1, **kw})) == code


def test_linear_calls():
    assert L.rn_linear_attention_workspace_bytes(None) == 0
    assert chunked(lin(N=0)) == INV and chunked(lin(N=(1 << 30) + 1, out_stride=(1 << 40, 64, 512))) == UNS
    assert step(lin()) == INV                                        # N != 1
    assert step(lin(N=1, T=5)) == INV and step(lin(N=1), state=None) == INV
    assert step(lin(N=1), state=FAKE + 4) == INV and step(lin(N=1), slots=FAKE) == INV     # n_slots = 0
    assert step(lin(N=1, n_slots=4), slots=FAKE + 2) == INV
    assert step(lin(N=1), q=None) == INV and step(lin(N=1), out=FAKE + 1) == INV
    d = lin()
    for kw in (dict(cu=FAKE), dict(lens=FAKE + 1), dict(slots=FAKE), dict(q=None), dict(g=None), dict(g=FAKE + 2),
               dict(s0=FAKE + 8), dict(s1=FAKE + 8), dict(out=None)):
        assert chunked(d, **kw) == INV, kw
    packed = lin(T=200, S=3)
    assert chunked(packed) == INV                                    # no cu_seqlens
    assert chunked(packed, cu=FAKE, lens=FAKE) == INV
    assert chunked(lin(T=99), cu=FAKE) == INV                        # N > T
    long = lin(N=1 << 16, q_stride=(1 << 30, 64, 512), out_stride=(1 << 30, 64, 512))
    need = L.rn_linear_attention_workspace_bytes(ctypes.byref(long))
    assert need > 0
    assert chunked(long, n=need - 1) == WS and chunked(long, ws=None) == WS and chunked(long, ws=FAKE + 16) == INV


def test_workspace_size_passes_32_bits():
    """A million tokens of 128 heads: sizes are formed in 64 bits."""
    d = lin(S=64, N=1 << 20, H=128, H_q=128, H_k=128, H_v=128, d_k=256, d_v=512, flags=rn.RN_LINEAR_GENERIC,
            out_stride=(1 << 40, 512, 512 * 128))
    a = L.rn_linear_attention_workspace_bytes(ctypes.byref(d))
    assert a % 256 == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        rn.rn_layernorm(x)
    with pytest.raises(ValueError):
        rn.rn_layernorm_backward(x, x)
    with pytest.raises(ValueError):
        rn.rn_rotary(torch.zeros(1, 2, 3, 8), None, np.ones(4))
    z = torch.zeros(1, 2, 3, 8)
    with pytest.raises(ValueError):
        rn.rn_linear_attention_chunked(z, z, z, torch.zeros(1, 2, 3))
    with pytest.raises(ValueError):
        rn.rn_linear_attention_step(z, z, z, torch.zeros(1, 2, 3), torch.zeros(1, 2, 8, 8))


def test_outputs_that_are_other_inputs_are_refused():
    """Blocks read what others would overwrite: an output that is another operand's input."""
    d = rot()
    assert rotary(d, q=FAKE, k=2 * FAKE, qo=2 * FAKE) == INV and b"own input" in L.rn_last_error()
    assert rotary(d, q=FAKE, k=2 * FAKE, ko=FAKE) == INV and b"own input" in L.rn_last_error()
    d = lin()
    for kw in (dict(out=FAKE), dict(q=5 * FAKE, out=FAKE)):         # (k and v are FAKE)
        assert chunked(d, **kw) == INV and b"must not be q, k or v" in L.rn_last_error()
    assert step(lin(N=1), q=5 * FAKE, out=5 * FAKE) == INV and b"must not be q, k or v" in L.rn_last_error()


@pytest.mark.parametrize("generic", [0, rn.RN_LINEAR_GENERIC])
def test_packed_workspace_does_not_grow_with_the_sequences(generic):
    """The states kept between passes are those of segments, of which a fixed number of tokens has a
    bounded number, however many sequences share them."""
    T = 1 << 20

    def need(S, N=T):
        return L.rn_linear_attention_workspace_bytes(ctypes.byref(lin(S=S, N=N, T=T, d_k=256, d_v=512, flags=generic,
                                                                           out_stride=(0, 512, 4096))))

    few = need(1)                     # one sequence: a state for each segment
    assert few > 0
    for S in (2, 30, 1000, 20000, 65534):
        assert 0 < need(S) <= 2 * few + 4096, S
    for N in (T // 50, T // 500, 1000):   # a bound on the lengths, in a buffer with room for many more
        for S in (1, 3, 100, 1000, 20000):
            assert need(S, N) <= 2 * few + 4096, (S, N)


def test_header_limits_are_the_calls_limits():
    """The largest sizes that the header gives for linear attention are taken, the next ones are not."""
    import pathlib
    import re
    text = (pathlib.Path(__file__).parent.parent / "include" / "rn_retention.h").read_text()
    text = text[text.index("typedef struct rn_linear_desc"):text.index("} rn_linear_desc;")]
    wide = dict(out_stride=(1 << 40, 1 << 24, 512), q_stride=(0, 0, 0), k_stride=(0, 0, 0), v_stride=(0, 0, 0), N=1, H=1,
                H_q=1, H_k=1, H_v=1)
    for field in ("S", "H", "d_k", "d_v"):
        most = int(re.search(r"\b%s;[^\n]*?1 \.\. (\d+)" % field, text).group(1))
        for n, code in ((most, INV), (most + 1, UNS)):       # (a NULL pointer, once the sizes are taken)
            assert chunked(lin(**{**wide, field: n}), q=None) == code, (field, n)


def test_workspace_bytes():
    """The exact need of a known shape, and a bound that holds for all: a pass cuts the tokens so that
    about 256 to 768 blocks of at most 64 KiB of state (128 KiB for 128 columns) run at once; rests of
    segments and the room that ragged lengths need multiply that by at most 8."""
    d = lin(S=1, N=8192, H=16, H_q=16, H_k=16, H_v=16, d_k=256, d_v=512, q_stride=(0, 256, 4096), k_stride=(0, 256, 4096),
            v_stride=(0, 512, 8192), out_stride=(0, 512, 8192))
    # 64 blocks a segment on 256 compute units: four segments of 2048 tokens
    assert L.rn_linear_attention_workspace_bytes(ctypes.byref(d)) == 4 * 16 * 256 * 512 * 4 + 256
    rng = np.random.default_rng(41)
    seen = 0
    for _ in range(4000):
        S, N = (int(2 ** rng.uniform(0, b)) for b in (15.9, 30))
        H = int(2 ** rng.uniform(0, 10))
        dk, dv = int(rng.integers(1, 257)), int(rng.integers(1, 513))
        packed = rng.random() < 0.6
        T = min(N * int(2 ** rng.uniform(0, 12)), (1 << 31) - 1) if packed else 0
        st = (0, 1 << 10, 1 << 20) if packed else (1 << 40, 0 if H == 1 else dv, H * dv)
        if not packed and N * H * dv > 1 << 40:
            continue
        need = L.rn_linear_attention_workspace_bytes(ctypes.byref(lin(
            S=S, N=N, T=T, H=H, H_q=1, H_k=1, H_v=1, d_k=dk, d_v=dv, out_stride=st, flags=int(rng.choice([0, rn.RN_LINEAR_GENERIC])))))
        assert need <= 8 * 768 * (64 << 10) + (1 << 20), (S, N, H, dk, dv, T)
        seen += need > 0
    assert seen > 100


def test_outputs_that_partly_overlap_are_refused():
    """Rows or heads shifted by less than apart; views that interleave without meeting stay allowed
    (such calls fail for the reason put into them: an unknown flag or a missing pointer)."""
    B = 1 << 20
    d = norm(rows=1000)                                                # 1000 rows of 64 bf16, 128 bytes apart
    for shift in (2, 126, 128, -128, 999 * 128, -999 * 128 + 126):
        assert norm_forward(d, x=B, out=B + shift) == INV and b"out overlaps x" in L.rn_last_error(), shift
        assert norm_forward(d, x=B, r=4 * B, s=4 * B + shift, out=8 * B) == INV and b"sum_out overlaps residual" in L.rn_last_error()
        assert norm_backward(d, dout=B, x=4 * B, dx=B + shift) == INV and b"dx overlaps dout" in L.rn_last_error()
        assert norm_backward(d, dout=B, x=4 * B, dx=4 * B + shift) == INV and b"dx overlaps x" in L.rn_last_error()
    assert norm_forward(d, x=B, out=8 * B, s=8 * B + 2) == INV and b"out overlaps sum_out" in L.rn_last_error()
    wide = norm(rows=1000, x_stride=160, out_stride=160, sum_stride=160)
    for shift in (128, 192, -128, 320 * 1000, 320 * 999 + 128, -320 * 1000):      # columns beside x's own, or rows behind
        assert norm_backward(wide, dout=4 * B, x=B, dx=B + shift, ws=None) == WS, shift
    for shift in (126, 194, -126, 320 + 126, 320 * 999 - 126):
        assert norm_backward(wide, dout=4 * B, x=B, dx=B + shift, ws=None) == INV and b"dx overlaps x" in L.rn_last_error(), shift
    # heads of one projection [2, 100, 12 heads of 128]: q has eight of them, k four
    s = (12 * 128 * 100, 128, 12 * 128)
    d = rot(B=2, N=100, H_k=4, q_stride=s, k_stride=s, q_out_stride=s, k_out_stride=s)
    args = dict(q=B, k=B + 8 * 256, qo=16 * B, ko=32 * B)
    for kw, text in ((dict(qo=B + 256), b"q_out overlaps q"), (dict(qo=B + 24 * 128 * 7 + 6), b"q_out overlaps q"),
                     (dict(qo=B + 9 * 256), b"q_out overlaps q"), (dict(ko=B + 7 * 256), b"k_out overlaps"),
                     (dict(qo=16 * B, ko=16 * B + 256), b"q_out overlaps k_out")):
        assert rotary(d, **{**args, **kw}) == INV and text in L.rn_last_error(), kw
    # linear attention: out among the heads of v's buffer
    s = (0, 64, 1024)
    one = dict(S=1, N=1 << 12, H=4, H_q=4, H_k=4, H_v=4, q_stride=s, k_stride=s, v_stride=s, out_stride=s, flags=rn.RN_LINEAR_GENERIC)
    d = lin(**one)
    assert L.rn_linear_attention_workspace_bytes(ctypes.byref(d)) > 0
    f = lambda q, k, v, out: L.rn_linear_attention_chunked(  # noqa: E731
        ctypes.byref(d), None, None, None, q, k, v, FAKE, None, None, out, 1 << 30, 1 << 40, None)
    q, k, v = B, B + 4 * 128, B + 8 * 128
    for out, text in ((B + 128, b"out overlaps q"), (B + 5 * 128, b"out overlaps k"), (B + 9 * 128, b"out overlaps v"),
                      (B - 128, b"out overlaps q"), (B + 2048 * 50 + 130, b"out overlaps q")):
        assert f(q, k, v, out) == INV and text in L.rn_last_error(), out


def test_overlap_of_strided_boxes_against_sets_of_addresses():
    """The layer norm's and rotary's refusals against the sets of elements that the views have."""
    rng = np.random.default_rng(42)
    cells = lambda n, s, d: (np.add.outer(np.add.outer(np.add.outer(np.arange(n[0]) * s[0], np.arange(n[1]) * s[1]),  # noqa: E731
                                                       np.arange(n[2]) * s[2]), np.arange(d))).ravel()
    base, hit, clear = 1 << 20, 0, 0
    for _ in range(3000):
        n, d = [int(x) for x in rng.integers(1, 5, 3)], 2 * int(rng.integers(1, 4))
        order, s, span = rng.permutation(3), [0, 0, 0], d
        for a in order:
            s[a] = span + int(rng.integers(0, 4)) * int(rng.integers(0, 6))
            span = s[a] * n[a]
        diff = int(rng.integers(-span - d, span + d + 1))
        if diff == 0:
            continue
        own = cells(n, s, d)
        meet = bool(np.intersect1d(own, own + diff).size)
        desc = rot(B=n[0], H_q=n[1], H_k=0, N=n[2], d=d, rot=2, q_stride=tuple(s), q_out_stride=tuple(s), dtype=1)
        # (a call that is not refused for its overlap would launch: an unaligned pos is found before it)
        code = L.rn_rotary(ctypes.byref(desc), None, base, None, base + 2 * diff, None, None) if meet else None
        if meet:
            assert code == INV and b"q_out overlaps q" in L.rn_last_error(), (n, s, d, diff)
            hit += 1
        else:
            nd = norm(rows=n[2], d=d, x_stride=s[2], sum_stride=s[2], out_stride=s[2])
            m1 = bool(np.intersect1d(cells((1, 1, n[2]), s, d), cells((1, 1, n[2]), s, d) + diff).size)
            got = norm_backward(nd, dout=1 << 24, x=base, dx=base + 2 * diff, ws=None)
            assert got == (INV if m1 or (n[2] > 1 and s[2] < d) else WS), (n, s, d, diff)
            clear += got == WS
    assert hit > 300 and clear > 300


def test_a_replaced_base_has_to_be_finite():
    """Past the largest number it would turn every pair but the first by nothing."""
    with pytest.raises(rn.RnError):
        rn.rn_rotary_frequencies(4, kind="base", factor=1e200)
    with pytest.raises(rn.RnError):
        rn.rn_rotary_frequencies(128, kind="base", factor=1e306)
    theta, _ = rn.rn_rotary_frequencies(128, kind="base", factor=1e290)
    assert np.abs(theta / (1e4 * 1e290 ** (128 / 126)) ** (-np.arange(64) / 64) - 1).max() < 1e-12
