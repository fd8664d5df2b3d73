"""The short causal convolution and the selective scan: prompts, single tokens, gradients.

As the operators around retention (block_ops.py): the functions carry the C names and only marshal
arguments. Tensors of tokens are [B, N, D] (B and C of the scan [B, G, N, n]) with any strides as long
as their last axis is contiguous; calls run on the current stream of their tensors' device. New outputs
are allocated with torch.

A batch is padded (``lengths`` device int32 [B], or None: all of N) or packed (B = 1 and
``cu_seqlens`` device int32 [S + 1], first entry 0). ``max_len``: no sequence is longer (host number;
longer ones are cut). Rows of no sequence are not read, and not written (zero in a new output).
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import lib
from .block_ops import _call, _code, _device, _get_workspace, _int32, _p, _whole

RN_SEQ_ZERO_REST, RN_CONV_SILU, RN_SCAN_SOFTPLUS = 1, 2, 2

_i32, _i64, _u32, _vp, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t


class RnConvDesc(ctypes.Structure):
    _fields_ = [("S", _i32), ("N", _i32), ("D", _i32), ("K", _i32), ("dtype", _i32), ("flags", _u32), ("T", _i64),
                ("n_slots", _i32), ("x_stride", _i64 * 2), ("out_stride", _i64 * 2), ("dx_stride", _i64 * 2)]


class RnScanDesc(ctypes.Structure):
    _fields_ = [("S", _i32), ("N", _i32), ("D", _i32), ("n", _i32), ("G", _i32), ("dtype", _i32), ("flags", _u32),
                ("n_slots", _i32), ("T", _i64), ("x_stride", _i64 * 2), ("dt_stride", _i64 * 2),
                ("z_stride", _i64 * 2), ("out_stride", _i64 * 2), ("b_stride", _i64 * 3), ("c_stride", _i64 * 3)]


class RnScanGradDesc(ctypes.Structure):
    _fields_ = [("dx_stride", _i64 * 2), ("ddt_stride", _i64 * 2), ("dz_stride", _i64 * 2), ("db_stride", _i64 * 3),
                ("dc_stride", _i64 * 3)]


_pack_conv = struct.Struct("@iiiiiIqi6q").pack
_pack_scan = struct.Struct("@iiiiiiIiq14q").pack
_pack_grads = struct.Struct("@12q").pack
assert struct.calcsize("@iiiiiIqi6q") == ctypes.sizeof(RnConvDesc)
assert struct.calcsize("@iiiiiiIiq14q") == ctypes.sizeof(RnScanDesc)
assert struct.calcsize("@12q") == ctypes.sizeof(RnScanGradDesc)


def _bind(L):
    for name, args, res in (
            ("rn_short_conv", [_vp] * 11, _i32),
            ("rn_short_conv_step", [_vp] * 8, _i32),
            ("rn_short_conv_backward_workspace_bytes", [_vp], _sz),
            ("rn_short_conv_backward", [_vp] * 14 + [_sz, _vp], _i32),
            ("rn_selective_scan_workspace_bytes", [_vp], _sz),
            ("rn_selective_scan_chunked", [_vp] * 16 + [_sz, _vp], _i32),
            ("rn_selective_scan_step", [_vp] * 13, _i32),
            ("rn_selective_scan_backward_workspace_bytes", [_vp], _sz),
            ("rn_selective_scan_backward", [_vp] * 25 + [_sz, _vp], _i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


_bind(lib)


# ---- batches of sequences -------------------------------------------------------------------

def _tokens(t, name):
    """Strides (sequence, token) of [B, N, D] with a contiguous last axis."""
    s = t.stride()
    if len(s) != 3:
        raise ValueError(f"{name} must be [B, N, D]; got {tuple(t.shape)}")
    if s[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return s[:2]


def _same(t, x, name):
    if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
        raise ValueError(f"{name} must be {x.dtype} {tuple(x.shape)}; got {t.dtype} {tuple(t.shape)}")


def _batch(x, lengths, cu, max_len):
    """(S, N, T) of a batch whose token rows are x's, its lists checked."""
    if x.dim() != 3 or x.numel() == 0:
        raise ValueError(f"x must be [B, N, D] and not empty; got {tuple(x.shape)}")
    B, rows = x.shape[0], x.shape[1]
    if cu is not None:
        if B != 1 or lengths is not None or cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("a packed batch is [1, T, D] with cu_seqlens [S + 1] and without lengths")
        S, T, N = cu.numel() - 1, rows, rows
        _int32(cu, S + 1, "cu_seqlens")
    else:
        S, T, N = B, 0, rows
        _int32(lengths, S, "lengths")
    if max_len is not None:
        if not 1 <= max_len <= N:
            raise ValueError(f"max_len={max_len} outside [1, {N}]")
        N = max_len
    return S, N, T


def _rest(new, rows, N, T, lengths):
    """The flag that zeroes rows of no sequence in new outputs, and those past N of a padded batch
    here."""
    if not new or (T == 0 and lengths is None and N == rows):
        return 0
    if T == 0 and N < rows:
        for t in new:
            t[..., N:, :].zero_()
    return RN_SEQ_ZERO_REST


def _states(state_in, state_out, slots, S, row, dtype, like):
    """(state_out, slots a buffer) with the buffers checked; state_out may be True: a new one."""
    _int32(slots, S, "slots")
    if slots is not None and state_out is True:
        raise ValueError("with slots, state_out must be a tensor")
    if state_out is True:
        state_out = like.new_empty((S, *row), dtype=dtype)
    elif state_out is False:
        state_out = None
    n = None
    for s, name in ((state_in, "state_in"), (state_out, "state_out")):
        if s is None:
            continue
        if s.dtype != dtype or not s.is_contiguous() or s.dim() != 1 + len(row) or s.shape[1:] != row or \
                s.shape[0] < 1 or (slots is None and s.shape[0] != S):
            raise ValueError(f"{name} must be contiguous {dtype} {('slots' if slots is not None else S, *row)}; got "
                             f"{s.dtype} {tuple(s.shape)}")
        if slots is not None and n not in (None, s.shape[0]):
            raise ValueError("state_in and state_out must have the same number of slots")
        n = s.shape[0]
    return state_out, n or 1


# ---- short convolution ----------------------------------------------------------------------

def _conv_weight(D, weight, bias):
    shape = weight.shape
    if len(shape) != 2 or shape[0] != D:
        raise ValueError(f"weight must be [{D}, K]; got {tuple(shape)}")
    _whole(weight, torch.float32, shape, "weight")
    if bias is not None:
        _whole(bias, torch.float32, (D,), "bias")
    return shape[1]


def _state_pool(state, slots, S, row, dtype):
    """The number of states in the buffer of a step."""
    if slots is not None:
        _int32(slots, S, "slots")
    shape = state.shape
    if state.dtype != dtype or len(shape) != 3 or shape[1:] != row or not state.is_contiguous() or shape[0] < 1 or \
            (slots is None and shape[0] != S):
        raise ValueError(f"state must be contiguous {dtype} {('slots' if slots is not None else S, *row)}; got {state.dtype} "
                         f"{tuple(shape)}")
    return shape[0]


def rn_short_conv(x, weight, bias=None, *, silu=False, lengths=None, cu_seqlens=None, max_len=None, state_in=None,
                  state_out=None, slots=None, out=None):
    """Causal convolution of every channel of x [B, N, D] with its own weights (float32 [D, K], K <= 8)
    and bias (float32 [D] or None): u_t = bias + sum_j weight[:, j] x_{t-K+1+j}; returns (out, state_out)
    with out = u, or u sigmoid(u) with ``silu``.

    The K - 1 inputs before a sequence's first token are its state: state_in, state_out of x's type
    [S, K - 1, D], or pools [slots, K - 1, D] with ``slots`` device int32 [S] (distinct; -1: start from
    zeros, keep nothing); None: start from zeros / discard; state_out may be True (new; not with slots) or
    state_in itself."""
    dev = _device(x, weight, bias, lengths, cu_seqlens, slots, out, state_in,
                  state_out if isinstance(state_out, torch.Tensor) else None)
    S, N, T = _batch(x, lengths, cu_seqlens, max_len)
    D = x.shape[2]
    K = _conv_weight(D, weight, bias)
    state_out, n_slots = _states(state_in, state_out, slots, S, (K - 1, D), x.dtype, x)
    flags = RN_CONV_SILU if silu else 0
    if out is None:
        out = x.new_empty(x.shape)
        flags |= _rest((out,), x.shape[1], N, T, lengths)
    else:
        _same(out, x, "out")
    desc = _pack_conv(S, N, D, K, _code(x.dtype), flags, T, n_slots, *_tokens(x, "x"), *_tokens(out, "out"), 0, 0)
    _call(dev, lib.rn_short_conv, desc, _p(cu_seqlens), _p(lengths), _p(slots), x.data_ptr(), weight.data_ptr(), _p(bias),
          _p(state_in), _p(state_out), out.data_ptr())
    return out, state_out


def rn_short_conv_step(x, weight, bias, state, *, silu=False, slots=None, out=None):
    """One token for each of S sequences: x [S, 1, D]; ``state`` (of x's type [S, K - 1, D], or a pool with
    ``slots``) is updated in place. Returns out [S, 1, D]; a sequence with slot -1 is skipped, its row of
    out set to zero."""
    dev = _device(x, weight, bias, state, slots, out)
    shape, kind = x.shape, x.dtype
    if len(shape) != 3 or shape[1] != 1 or 0 in shape:
        raise ValueError(f"the step takes one token a sequence: x [S, 1, D]; got {tuple(shape)}")
    S, _, D = shape
    K = _conv_weight(D, weight, bias)
    n_slots = _state_pool(state, slots, S, (K - 1, D), kind)
    if out is None:
        out, os = x.new_empty(shape), (D, D)
    else:
        _same(out, x, "out")
        os = _tokens(out, "out")
    desc = _pack_conv(S, 1, D, K, _code(kind), RN_CONV_SILU if silu else 0, 0, n_slots, *_tokens(x, "x"), *os, 0, 0)
    _call(dev, lib.rn_short_conv_step, desc, _p(slots), x.data_ptr(), weight.data_ptr(), _p(bias), state.data_ptr(),
          out.data_ptr())
    return out


def _grad_state(t, S, row, name):
    _whole(t, torch.float32, (S, *row), name)


def rn_short_conv_backward_workspace_bytes(x, weight, *, cu_seqlens=None, max_len=None) -> int:
    """Bytes of workspace ``rn_short_conv_backward`` needs for these tensors."""
    S, N, T = _batch(x, None, cu_seqlens, max_len)
    st = _tokens(x, "x")
    desc = _pack_conv(S, N, x.shape[2], weight.shape[1], _code(x.dtype), 0, T, 0, *st, *st,
                      x.shape[1] * x.shape[2], x.shape[2])
    return int(lib.rn_short_conv_backward_workspace_bytes(desc))


def rn_short_conv_backward(dout, x, weight, bias=None, *, silu=False, lengths=None, cu_seqlens=None, max_len=None,
                           state_in=None, dstate_out=None, dx=None, want_dweight=True, want_dstate_in=False,
                           workspace=None):
    """Gradients of ``rn_short_conv`` (same arguments; states per sequence, without slots) given those of
    its output and, optionally, of its final state (``dstate_out``, float32 [S, K - 1, D]). Returns a dict
    with dx (x's type) and, where wanted, dweight and dbias (float32; dbias where there is a bias) and
    dstate_in (float32)."""
    dev = _device(x, dout, weight, bias, lengths, cu_seqlens, state_in, dstate_out, dx, workspace)
    S, N, T = _batch(x, lengths, cu_seqlens, max_len)
    _same(dout, x, "dout")
    D = x.shape[2]
    K = _conv_weight(D, weight, bias)
    row = (K - 1, D)
    _states(state_in, None, None, S, row, x.dtype, x)
    _grad_state(dstate_out, S, row, "dstate_out")
    flags = RN_CONV_SILU if silu else 0
    if dx is None:
        dx = x.new_empty(x.shape)
        flags |= _rest((dx,), x.shape[1], N, T, lengths)
    else:
        _same(dx, x, "dx")
    got = {"dx": dx}
    if want_dweight:
        got["dweight"] = torch.empty_like(weight)
        if bias is not None:
            got["dbias"] = torch.empty_like(bias)
    if want_dstate_in:
        got["dstate_in"] = x.new_empty((S, *row), dtype=torch.float32)
    desc = _pack_conv(S, N, D, K, _code(x.dtype), flags, T, 0, *_tokens(x, "x"), *_tokens(dout, "dout"), *_tokens(dx, "dx"))
    if want_dweight:
        workspace = _get_workspace(workspace, lib.rn_short_conv_backward_workspace_bytes(desc), x)
    else:
        workspace = None
    _call(dev, lib.rn_short_conv_backward, desc, _p(cu_seqlens), _p(lengths), dout.data_ptr(), x.data_ptr(),
          weight.data_ptr(), _p(bias), _p(state_in), _p(dstate_out), dx.data_ptr(), _p(got.get("dweight")),
          _p(got.get("dbias")), _p(got.get("dstate_in")), _p(workspace), 0 if workspace is None else workspace.numel())
    return got


# ---- selective scan -------------------------------------------------------------------------

def _groups(t, x, n, name):
    """Strides (sequence, group, token) of [B, G, N, n] with a contiguous last axis."""
    if t.dim() != 4 or t.dtype != x.dtype or t.shape[0] != x.shape[0] or t.shape[2] != x.shape[1] or t.shape[3] != n:
        raise ValueError(f"{name} must be {x.dtype} [{x.shape[0]}, G, {x.shape[1]}, {n}]; got {t.dtype} {tuple(t.shape)}")
    s = t.stride()
    if s[3] != 1 and n > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return s[:3]


def _scan_tensors(x, dt, A, B, C, D, dt_bias, z):
    """Checks what the scan's calls share; returns the states a channel, groups, and the strides."""
    d = x.shape[2]
    if A.dim() != 2 or A.shape[0] != d:
        raise ValueError(f"A must be [{d}, n]; got {tuple(A.shape)}")
    _whole(A, torch.float32, A.shape, "A")
    n = A.shape[1]
    _same(dt, x, "dt")
    _same(z, x, "z")
    bs, cs = _groups(B, x, n, "B"), _groups(C, x, n, "C")
    if B.shape != C.shape:
        raise ValueError(f"B and C must have the same shape; got {tuple(B.shape)}, {tuple(C.shape)}")
    _whole(D, torch.float32, (d,), "D")
    _whole(dt_bias, torch.float32, (d,), "dt_bias")
    return n, B.shape[1], (*_tokens(x, "x"), *_tokens(dt, "dt"), *((0, 0) if z is None else _tokens(z, "z"))), (*bs, *cs)


def _scan_desc(S, N, T, x, n, G, flags, n_slots, tokens, out, groups):
    return _pack_scan(S, N, x.shape[2], n, G, _code(x.dtype), flags, n_slots, T, *tokens, *out, *groups)


def rn_selective_scan_workspace_bytes(x, A, B, *, cu_seqlens=None, max_len=None) -> int:
    """Bytes of workspace ``rn_selective_scan_chunked`` needs for these tensors."""
    S, N, T = _batch(x, None, cu_seqlens, max_len)
    return int(lib.rn_selective_scan_workspace_bytes(
        _scan_desc(S, N, T, x, A.shape[1], B.shape[1], 0, 0, (0,) * 6, (0, 0), (0,) * 6)))


def rn_selective_scan_chunked(x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, z=None, lengths=None,
                              cu_seqlens=None, max_len=None, state_in=None, state_out=None, slots=None, out=None,
                              workspace=None):
    """Selective scan over prompts: with D_t = softplus(dt_t + dt_bias) (or dt_t + dt_bias without
    ``softplus``), h_t = exp(D_t A) h_{t-1} + D_t x_t B_t, y_t = C_t h_t + D x_t; returns (out, state_out)
    with out = y, or y z sigmoid(z) where z is given.

    x, dt, z [B, N, D] and B, C [B, G, N, n] of one type (G divides D: channels of a group share them);
    A float32 [D, n]; D, dt_bias float32 [D] or None. state_in, state_out: float32 [S, D, n], or pools
    [slots, D, n] with ``slots`` device int32 [S] (distinct; -1: start from zeros, keep nothing); None:
    start from zeros / discard; state_out may be True (new; not with slots) or state_in itself."""
    dev = _device(x, dt, A, B, C, D, dt_bias, z, lengths, cu_seqlens, slots, out, workspace, state_in,
                  state_out if isinstance(state_out, torch.Tensor) else None)
    S, N, T = _batch(x, lengths, cu_seqlens, max_len)
    n, G, tokens, groups = _scan_tensors(x, dt, A, B, C, D, dt_bias, z)
    state_out, n_slots = _states(state_in, state_out, slots, S, (x.shape[2], n), torch.float32, x)
    flags = RN_SCAN_SOFTPLUS if softplus else 0
    if out is None:
        out = x.new_empty(x.shape)
        flags |= _rest((out,), x.shape[1], N, T, lengths)
    else:
        _same(out, x, "out")
    desc = _scan_desc(S, N, T, x, n, G, flags, n_slots, tokens, _tokens(out, "out"), groups)
    workspace = _get_workspace(workspace, lib.rn_selective_scan_workspace_bytes(desc), x)
    _call(dev, lib.rn_selective_scan_chunked, desc, _p(cu_seqlens), _p(lengths), _p(slots), x.data_ptr(), dt.data_ptr(),
          A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(dt_bias), _p(z), _p(state_in), _p(state_out), out.data_ptr(),
          _p(workspace), 0 if workspace is None else workspace.numel())
    return out, state_out


def rn_selective_scan_step(x, dt, A, B, C, state, D=None, *, dt_bias=None, softplus=True, z=None, slots=None, out=None):
    """One token for each of S sequences: x, dt, z [S, 1, D], B, C [S, G, 1, n] as in
    ``rn_selective_scan_chunked``; ``state`` (float32 [S, D, n], or a pool with ``slots``) is updated in
    place. Returns out [S, 1, D]; a sequence with slot -1 is skipped, its row of out set to zero."""
    dev = _device(x, dt, A, B, C, D, dt_bias, z, state, slots, out)
    shape = x.shape
    if len(shape) != 3 or shape[1] != 1 or 0 in shape:
        raise ValueError(f"the step takes one token a sequence: x [S, 1, D]; got {tuple(shape)}")
    S = shape[0]
    n, G, tokens, groups = _scan_tensors(x, dt, A, B, C, D, dt_bias, z)
    n_slots = _state_pool(state, slots, S, (shape[2], n), torch.float32)
    if out is None:
        out = x.new_empty(x.shape)
    else:
        _same(out, x, "out")
    desc = _scan_desc(S, 1, 0, x, n, G, RN_SCAN_SOFTPLUS if softplus else 0, n_slots, tokens, _tokens(out, "out"), groups)
    _call(dev, lib.rn_selective_scan_step, desc, _p(slots), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
          C.data_ptr(), _p(D), _p(dt_bias), _p(z), state.data_ptr(), out.data_ptr())
    return out


def rn_selective_scan_backward_workspace_bytes(x, A, B, *, cu_seqlens=None, max_len=None) -> int:
    """Bytes of workspace ``rn_selective_scan_backward`` needs for these tensors."""
    S, N, T = _batch(x, None, cu_seqlens, max_len)
    return int(lib.rn_selective_scan_backward_workspace_bytes(
        _scan_desc(S, N, T, x, A.shape[1], B.shape[1], 0, 0, (0,) * 6, (0, 0), (0,) * 6)))


def rn_selective_scan_backward(dout, x, dt, A, B, C, D=None, *, dt_bias=None, softplus=True, z=None, lengths=None,
                               cu_seqlens=None, max_len=None, state_in=None, dstate_out=None, want_dstate_in=False,
                               dx=None, ddt=None, dB=None, dC=None, dz=None, workspace=None):
    """Gradients of ``rn_selective_scan_chunked`` (same arguments; states per sequence, without slots) given
    those of its output and, optionally, of its final state (``dstate_out``, float32 [S, D, n]). Returns a
    dict with dx, ddt, dB, dC (x's type; new, or those given, whose rows of no sequence are not written),
    dA (float32) and, where there is a z, D or dt_bias, dz (x's type), dD and ddt_bias (float32); with
    ``want_dstate_in`` dstate_in (float32 [S, D, n])."""
    dev = _device(x, dout, dt, A, B, C, D, dt_bias, z, lengths, cu_seqlens, state_in, dstate_out, dx, ddt, dB, dC, dz,
                  workspace)
    S, N, T = _batch(x, lengths, cu_seqlens, max_len)
    _same(dout, x, "dout")
    n, G, tokens, groups = _scan_tensors(x, dt, A, B, C, D, dt_bias, z)
    row = (x.shape[2], n)
    _states(state_in, None, None, S, row, torch.float32, x)
    _grad_state(dstate_out, S, row, "dstate_out")
    if dz is not None and z is None:
        raise ValueError("dz without z")
    got, new = {}, []
    for name, t, like in (("dx", dx, x), ("ddt", ddt, x), ("dB", dB, B), ("dC", dC, C), ("dz", dz, z)):
        if like is None:
            continue
        if t is None:
            t = x.new_empty(like.shape)
            new.append(t)
        else:
            _same(t, like, name)
        got[name] = t
    given = len(got) - len(new)
    rest = _rest(new, x.shape[1], N, T, lengths)
    if rest and given:                  # the call's zeros would reach the given ones too
        for t in new:
            t.zero_()
        rest = 0
    flags = rest | (RN_SCAN_SOFTPLUS if softplus else 0)
    got["dA"] = torch.empty_like(A)
    if D is not None:
        got["dD"] = torch.empty_like(D)
    if dt_bias is not None:
        got["ddt_bias"] = torch.empty_like(dt_bias)
    if want_dstate_in:
        got["dstate_in"] = x.new_empty((S, *row), dtype=torch.float32)
    desc = _scan_desc(S, N, T, x, n, G, flags, 0, tokens, _tokens(dout, "dout"), groups)
    grads = _pack_grads(*_tokens(got["dx"], "dx"), *_tokens(got["ddt"], "ddt"),
                        *((0, 0) if z is None else _tokens(got["dz"], "dz")), *_groups(got["dB"], x, n, "dB"),
                        *_groups(got["dC"], x, n, "dC"))
    workspace = _get_workspace(workspace, lib.rn_selective_scan_backward_workspace_bytes(desc), x)
    _call(dev, lib.rn_selective_scan_backward, desc, grads, _p(cu_seqlens), _p(lengths), dout.data_ptr(), x.data_ptr(),
          dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _p(D), _p(dt_bias), _p(z), _p(state_in), _p(dstate_out),
          got["dx"].data_ptr(), got["ddt"].data_ptr(), got["dA"].data_ptr(), got["dB"].data_ptr(), got["dC"].data_ptr(),
          _p(got.get("dD")), _p(got.get("ddt_bias")), _p(got.get("dz")), _p(got.get("dstate_in")), _p(workspace),
          0 if workspace is None else workspace.numel())
    return got
