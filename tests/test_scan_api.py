"""Host-side checks of the RMS norm, the short convolution and the selective scan (no GPU needed):
invalid arguments are rejected before any HIP call. Pointers passed here are never dereferenced."""
import ctypes
import math

import pytest
import torch

import linear_recurrent_sequence_rn_amd as rn

FAKE = 0x10000
L = rn.lib
INV, UNS, WS = rn.RN_ERR_INVALID_ARG, rn.RN_ERR_UNSUPPORTED, rn.RN_ERR_WORKSPACE
ref = ctypes.byref


def fill(cls, base, kw):
    d = cls()
    for name, v in {**base, **kw}.items():
        if isinstance(v, tuple):
            v = (ctypes.c_int64 * len(v))(*v)
        setattr(d, name, v)
    return d


def rms(**kw):
    return fill(rn.RnRmsDesc, dict(rows=4, d=64, in_dtype=1, out_dtype=1, group=0, eps=1e-5, x_stride=64, res_stride=64,
                                   sum_stride=64, out_stride=64, scale_stride=2), kw)


def forward(d, x=FAKE, r=None, w=None, s=None, out=2 * FAKE, scale=5 * FAKE):
    return L.rn_rmsnorm_forward(ref(d), x, r, w, s, out, scale, None)


def backward(d, dout=FAKE, x=FAKE, dx=2 * FAKE, dw=FAKE, ws=FAKE, n=1 << 40):
    return L.rn_rmsnorm_backward(ref(d), dout, x, None, None, dx, dw, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), INV), (dict(d=0), INV), (dict(d=16385), UNS), (dict(rows=(1 << 40) + 1), UNS), (dict(in_dtype=2), INV),
    (dict(in_dtype=3), INV), (dict(out_dtype=4), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(group=32), INV),
    (dict(out_dtype=2, group=48), UNS), (dict(out_dtype=3, group=-32), UNS), (dict(x_stride=-64), INV),
    (dict(scale_stride=(1 << 40) + 1), INV), (dict(out_stride=63), INV), (dict(sum_stride=10), INV),
    (dict(out_dtype=2, group=32, scale_stride=1), INV), (dict(out_dtype=3, scale_stride=0), INV)])
def test_rms_descriptors(kw, code):
    assert forward(rms(**kw), s=3 * FAKE) == code and L.rn_last_error() != b""


def test_rms_pointers_and_workspace():
    d = rms()
    assert L.rn_rmsnorm_forward(None, FAKE, None, None, None, FAKE, None, None) == INV
    assert forward(d, x=None) == INV and forward(d, out=None) == INV and forward(d, x=FAKE + 1) == INV
    assert forward(rms(out_dtype=2), scale=None) == INV and forward(rms(out_dtype=3), scale=FAKE + 2) == INV
    assert forward(rms(out_dtype=2), scale=2 * FAKE) == INV                  # scale and out the same
    assert forward(d, w=FAKE + 2) == INV
    assert forward(d, s=2 * FAKE) == INV                                     # out and sum_out the same
    assert forward(rms(out_dtype=2), out=FAKE) == INV                        # in place with other types
    assert forward(rms(out_stride=128), out=FAKE) == INV
    assert forward(d, out=FAKE + 64) == INV                                  # out overlaps x
    assert forward(d, s=FAKE + 64) == INV
    for dt in (2, 3):
        assert backward(rms(out_dtype=dt)) == INV                            # no gradient of 8 bits
        assert L.rn_rmsnorm_backward_workspace_bytes(ref(rms(out_dtype=dt))) == 0
    assert backward(d, dx=None) == INV and backward(d, dout=None) == INV and backward(d, dx=FAKE + 64) == INV
    need = L.rn_rmsnorm_backward_workspace_bytes(ref(d))
    assert need > 0 and backward(d, n=need - 1) == WS and backward(d, ws=None) == WS and backward(d, ws=FAKE + 16) == INV
    assert L.rn_rmsnorm_backward_workspace_bytes(None) == 0


def conv(**kw):
    s = (6400, 64)
    return fill(rn.RnConvDesc, dict(S=2, N=100, D=64, K=4, dtype=1, flags=0, T=0, n_slots=0, x_stride=s, out_stride=s,
                                    dx_stride=s), kw)


def run_conv(d, cu=None, lens=None, slots=None, x=FAKE, w=FAKE, b=None, s0=None, s1=None, out=1 << 30):
    return L.rn_short_conv(ref(d), cu, lens, slots, x, w, b, s0, s1, out, None)


def conv_step(d, slots=None, x=FAKE, w=FAKE, state=FAKE, out=1 << 30):
    return L.rn_short_conv_step(ref(d), slots, x, w, None, state, out, None)


def conv_back(d, cu=None, dout=FAKE, x=FAKE, w=FAKE, s0=None, ds1=None, dx=1 << 30, dw=FAKE, ds0=None, ws=FAKE, n=1 << 40):
    return L.rn_short_conv_backward(ref(d), cu, None, dout, x, w, None, s0, ds1, dx, dw, None, ds0, ws, n, None)


BATCH = [(dict(S=0), INV), (dict(N=0), INV), (dict(D=0), INV), (dict(S=65535), UNS), (dict(N=(1 << 30) + 1), UNS),
         (dict(D=65537), UNS), (dict(S=4096, N=1 << 20), UNS), (dict(dtype=2), INV), (dict(dtype=-1), INV), (dict(flags=4), INV),
         (dict(T=-1), INV), (dict(T=1 << 31), INV), (dict(x_stride=(-1, 64)), INV), (dict(out_stride=(6400, (1 << 40) + 1)), INV)]


@pytest.mark.parametrize("kw,code", BATCH + [
    (dict(K=0), INV), (dict(K=9), UNS), (dict(out_stride=(6400, 63)), INV), (dict(out_stride=(6399, 64)), INV)])
def test_conv_descriptors(kw, code):
    assert run_conv(conv(**kw)) == code and L.rn_last_error() != b""
    if "out_stride" not in kw:
        assert conv_step(conv(**{"N": 1, **kw})) == code or "N" in kw or kw == dict(S=4096, N=1 << 20)
        assert conv_back(conv(**kw)) == code and L.rn_short_conv_backward_workspace_bytes(ref(conv(**kw))) == 0
    else:
        assert conv_back(conv(dx_stride=kw["out_stride"])) == INV


def test_conv_calls():
    d = conv()
    assert L.rn_short_conv(None, None, None, None, FAKE, FAKE, None, None, None, FAKE, None) == INV
    for kw in (dict(cu=FAKE), dict(lens=FAKE + 1), dict(slots=FAKE), dict(x=None), dict(w=None), dict(out=None), dict(x=FAKE + 1),
               dict(w=FAKE + 2), dict(b=FAKE + 1), dict(s0=FAKE + 1), dict(s1=FAKE + 1), dict(out=FAKE), dict(out=FAKE + 128),
               dict(out=(1 << 30) + 1)):
        assert run_conv(d, **kw) == INV, kw
    packed = conv(T=200, S=3)
    assert run_conv(packed) == INV and run_conv(packed, cu=FAKE, lens=FAKE) == INV
    assert run_conv(conv(T=99), cu=FAKE) == INV                              # N > T
    assert run_conv(conv(n_slots=4), slots=FAKE + 2) == INV
    assert conv_step(d) == INV and conv_step(conv(N=1, T=5)) == INV and conv_step(conv(N=1), state=None) == INV
    assert conv_step(conv(N=1), slots=FAKE) == INV and conv_step(conv(N=1), out=FAKE) == INV
    assert conv_back(d, dout=None) == INV and conv_back(d, dx=None) == INV and conv_back(d, dx=FAKE) == INV
    assert conv_back(d, ds1=FAKE + 2) == INV and conv_back(d, ds1=FAKE, ds0=FAKE) == INV and conv_back(d, dw=FAKE + 2) == INV
    need = L.rn_short_conv_backward_workspace_bytes(ref(d))
    assert need > 0 and conv_back(d, n=need - 1) == WS and conv_back(d, ws=None) == WS and conv_back(d, ws=FAKE + 16) == INV


def scan(**kw):
    s, h = (6400, 64), (1600, 0, 16)
    return fill(rn.RnScanDesc, dict(S=2, N=100, D=64, n=16, G=1, dtype=1, flags=0, n_slots=0, T=0, x_stride=s, dt_stride=s,
                                    z_stride=s, out_stride=s, b_stride=h, c_stride=h), kw)


P = [FAKE * i for i in range(100, 110)]


def run_scan(d, cu=None, lens=None, slots=None, x=P[0], dt=P[1], A=P[2], B=P[3], C=P[4], skip=None, bias=None, z=None, s0=None,
             s1=None, out=1 << 30, ws=FAKE, n=1 << 40):
    return L.rn_selective_scan_chunked(ref(d), cu, lens, slots, x, dt, A, B, C, skip, bias, z, s0, s1, out, ws, n, None)


def scan_step(d, slots=None, x=P[0], state=FAKE, out=1 << 30):
    return L.rn_selective_scan_step(ref(d), slots, x, P[1], P[2], P[3], P[4], None, None, None, state, out, None)


SCAN = BATCH + [(dict(n=0), INV), (dict(n=65), UNS), (dict(G=0), INV), (dict(G=3), INV), (dict(b_stride=(0, -1, 0)), INV),
                (dict(c_stride=(0, 0, (1 << 40) + 1)), INV), (dict(dt_stride=(0, -1)), INV), (dict(z_stride=(-3, 0)), INV)]


@pytest.mark.parametrize("kw,code", SCAN)
def test_scan_descriptors(kw, code):
    assert run_scan(scan(**kw)) == code and L.rn_last_error() != b""
    assert L.rn_selective_scan_workspace_bytes(ref(scan(**kw))) == 0
    if "N" not in kw:
        assert scan_step(scan(**{"N": 1, **kw})) == code


def test_scan_calls():
    d = scan()
    assert L.rn_selective_scan_workspace_bytes(None) == 0
    for kw in (dict(cu=FAKE), dict(lens=FAKE + 1), dict(slots=FAKE), dict(x=None), dict(dt=None), dict(A=None), dict(B=None),
               dict(C=None), dict(out=None), dict(x=P[0] + 1), dict(A=P[2] + 2), dict(B=P[3] + 1), dict(skip=FAKE + 1),
               dict(bias=FAKE + 2), dict(z=FAKE + 1), dict(s0=FAKE + 8), dict(s1=FAKE + 8), dict(out=P[0]), dict(out=P[1]),
               dict(out=P[3]), dict(out=P[4]), dict(z=P[6], out=P[6]), dict(out=P[0] + 256)):
        assert run_scan(d, **kw) == INV, kw
    assert run_scan(scan(out_stride=(6400, 63))) == INV and run_scan(scan(out_stride=(0, 64))) == INV
    packed = scan(T=200, S=3)
    assert run_scan(packed) == INV and run_scan(packed, cu=FAKE, lens=FAKE) == INV
    assert run_scan(scan(T=99), cu=FAKE) == INV
    assert scan_step(d) == INV and scan_step(scan(N=1, T=5)) == INV and scan_step(scan(N=1), state=None) == INV
    assert scan_step(scan(N=1), state=FAKE + 4) == INV and scan_step(scan(N=1), slots=FAKE) == INV
    long = scan(N=1 << 14, S=1)
    need = L.rn_selective_scan_workspace_bytes(ref(long))
    assert need > 0 and run_scan(long, n=need - 1) == WS and run_scan(long, ws=None) == WS and run_scan(long, ws=FAKE + 16) == INV


def grads(**kw):
    s, h = (6400, 64), (1600, 1600, 16)
    return fill(rn.RnScanGradDesc, dict(dx_stride=s, ddt_stride=s, dz_stride=s, db_stride=h, dc_stride=h), kw)


Q = [FAKE * i for i in range(200, 212)]


def scan_back(d, g=grads(), cu=None, lens=None, dout=P[5], x=P[0], z=None, s0=None, ds1=None, dx=Q[0], ddt=Q[1], dA=Q[2], dB=Q[3],
              dC=Q[4], dskip=None, dbias=None, dz=None, ds0=None, ws=FAKE, n=1 << 40):
    return L.rn_selective_scan_backward(ref(d), ref(g) if g else None, cu, lens, dout, x, P[1], P[2], P[3], P[4], None, None, z, s0,
                                        ds1, dx, ddt, dA, dB, dC, dskip, dbias, dz, ds0, ws, n, None)


@pytest.mark.parametrize("kw,code", SCAN)
def test_scan_backward_descriptors(kw, code):
    assert scan_back(scan(**kw)) == code
    assert L.rn_selective_scan_backward_workspace_bytes(ref(scan(**kw))) == 0


def test_scan_backward_calls():
    d = scan()
    for kw in (dict(g=None), dict(cu=FAKE), dict(lens=FAKE + 1), dict(dout=None), dict(x=None), dict(dx=None), dict(ddt=None),
               dict(dA=None), dict(dB=None), dict(dC=None), dict(z=P[6]), dict(dz=Q[5]), dict(dx=Q[0] + 1), dict(dB=Q[3] + 1),
               dict(dA=Q[2] + 2), dict(dskip=FAKE + 2), dict(dbias=FAKE + 1), dict(s0=FAKE + 8), dict(ds1=FAKE + 4),
               dict(ds0=FAKE + 8), dict(ds0=FAKE, ds1=FAKE), dict(ds0=FAKE, s0=FAKE), dict(dx=P[0]), dict(ddt=P[1]), dict(dx=P[5]),
               dict(dB=P[3]), dict(dC=P[4]), dict(dx=Q[1]), dict(dC=Q[3]), dict(dC=Q[3] + 16), dict(dx=P[0] + 256),
               dict(z=P[6], dz=P[6]), dict(g=grads(dx_stride=(6400, 63))), dict(g=grads(ddt_stride=(-1, 64))),
               dict(g=grads(db_stride=(0, 0, 16))), dict(g=grads(dc_stride=(1600, 1600, 15))), dict(g=grads(dz_stride=(0, 0)), z=P[6], dz=Q[5])):
        assert scan_back(d, **kw) == INV, kw
    need = L.rn_selective_scan_backward_workspace_bytes(ref(d))
    assert need > 0 and scan_back(d, n=need - 1) == WS and scan_back(d, ws=None) == WS and scan_back(d, ws=FAKE + 16) == INV
    assert L.rn_selective_scan_backward_workspace_bytes(None) == 0


def test_workspace_sizes_pass_32_bits():
    d = scan(S=2048, N=1 << 20, D=64, x_stride=(1 << 40, 64), out_stride=(1 << 40, 64))
    d.S = 1
    d.N = 1 << 30
    assert L.rn_selective_scan_workspace_bytes(ref(d)) % 256 == 0
    wide = conv(D=65536, S=64, N=1 << 20, x_stride=(0, 0), dx_stride=(1 << 40, 65536), out_stride=(0, 0))
    assert L.rn_short_conv_backward_workspace_bytes(ref(wide)) == 128 * 5 * 65536 * 4


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 4, 64)
    w = torch.zeros(64, 4)
    for f in (lambda: rn.rn_rmsnorm(x), lambda: rn.rn_rmsnorm_backward(x, x), lambda: rn.rn_short_conv(x, w),
              lambda: rn.rn_short_conv_step(x[:, :1], w, None, torch.zeros(2, 3, 64)), lambda: rn.rn_short_conv_backward(x, x, w),
              lambda: rn.rn_selective_scan_chunked(x, x, w, x[:, None, :, :4], x[:, None, :, :4]),
              lambda: rn.rn_selective_scan_backward(x, x, x, w, x[:, None, :, :4], x[:, None, :, :4]),
              lambda: rn.rn_selective_scan_step(x[:, :1], x[:, :1], w, x[:, None, :1, :4], x[:, None, :1, :4], torch.zeros(2, 64, 4))):
        with pytest.raises(ValueError):
            f()


def test_states_shifted_against_each_other_are_refused():
    """A pool's first states as the start and its next ones as the result: one sequence would read what
    another one writes."""
    row = 3 * 64 * 2
    for off in (row, -row, 2, 2 * row - 2):
        assert run_conv(conv(), s0=FAKE, s1=FAKE + off) == INV and b"overlaps" in L.rn_last_error()
    for off in (16, 32 * row - 16):
        assert run_conv(conv(n_slots=32), slots=FAKE, s0=FAKE, s1=FAKE + off) == INV and b"overlaps" in L.rn_last_error()
    assert conv_back(conv(), ds0=FAKE, ds1=FAKE + 3 * 64 * 4) == INV and b"overlaps" in L.rn_last_error()
    row = 64 * 16 * 4
    for off in (row, -row, 16, 2 * row - 16):
        assert run_scan(scan(), s0=P[5], s1=P[5] + off) == INV and b"overlaps" in L.rn_last_error()
    assert run_scan(scan(n_slots=9), slots=FAKE, s0=P[5], s1=P[5] + 8 * row) == INV and b"overlaps" in L.rn_last_error()
    for kw in (dict(s0=P[5] + row), dict(ds1=P[5] + row), dict(ds1=P[5] - 16)):
        assert scan_back(scan(), ds0=P[5], dout=P[6], **kw) == INV and b"overlaps" in L.rn_last_error()
