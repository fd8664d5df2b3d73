"""The operators around retention: layer norm and root-mean-square norm (forward with the residual
sum, backward), rotary positions, and linear attention with a decay per head and token.

As the retention calls: the functions carry the C names and only marshal arguments. Tensors
may have any strides as long as their last axis is contiguous (a projection's output split
into heads needs no copy). Calls run on the current stream of their tensors' device; that
device need not be the current one. New outputs are allocated with torch.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import numpy as np
import torch

from . import RN_BF16, RN_E4M3, RN_F32, RN_INT8, _check, lib

RN_ROTARY_HALF, RN_ROTARY_INVERSE, RN_ROTARY_POS_TOKEN = 1, 2, 4
RN_ROPE_PLAIN, RN_ROPE_LINEAR, RN_ROPE_BASE, RN_ROPE_BY_PARTS = 0, 1, 2, 3
RN_LINEAR_ZERO_REST, RN_LINEAR_GENERIC = 1, 1 << 8

_i32, _i64, _f32, _f64, _vp, _sz = (ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                    ctypes.c_void_p, ctypes.c_size_t)


class RnNormDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("d", _i32), ("in_dtype", _i32), ("out_dtype", _i32), ("eps", _f32),
                ("x_stride", _i64), ("res_stride", _i64), ("sum_stride", _i64), ("out_stride", _i64)]


class RnRmsDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("d", _i32), ("in_dtype", _i32), ("out_dtype", _i32), ("group", _i32), ("eps", _f32),
                ("x_stride", _i64), ("res_stride", _i64), ("sum_stride", _i64), ("out_stride", _i64),
                ("scale_stride", _i64)]


class RnRotaryDesc(ctypes.Structure):
    _fields_ = [("B", _i32), ("N", _i32), ("H_q", _i32), ("H_k", _i32), ("d", _i32), ("rot", _i32),
                ("dtype", _i32), ("flags", ctypes.c_uint32), ("pos0", _i64), ("magnitude", _f32),
                ("theta", ctypes.c_void_p), ("q_stride", _i64 * 3), ("k_stride", _i64 * 3),
                ("q_out_stride", _i64 * 3), ("k_out_stride", _i64 * 3)]


class RnLinearDesc(ctypes.Structure):
    _fields_ = [("S", _i32), ("N", _i32), ("H", _i32), ("H_q", _i32), ("H_k", _i32), ("H_v", _i32),
                ("d_k", _i32), ("d_v", _i32), ("in_dtype", _i32), ("out_dtype", _i32),
                ("flags", ctypes.c_uint32), ("qk_scale", _f32), ("T", _i64), ("n_slots", _i32),
                ("q_stride", _i64 * 3), ("k_stride", _i64 * 3), ("v_stride", _i64 * 3),
                ("g_stride", _i64 * 3), ("out_stride", _i64 * 3)]


# The calls below fill their descriptors with struct, several times as fast as setting the
# fields one by one: a call costs the host a few microseconds in all, which is what the
# smallest ones take.
_pack_norm = struct.Struct("@qiiifqqqq").pack
_pack_rms = struct.Struct("@qiiiifqqqqq").pack
_pack_rotary = struct.Struct("@iiiiiiiIqfP12q").pack
_pack_linear = struct.Struct("@10iIfqi15q").pack
assert struct.calcsize("@qiiifqqqq") == ctypes.sizeof(RnNormDesc)
assert struct.calcsize("@qiiiifqqqqq") == ctypes.sizeof(RnRmsDesc)
assert struct.calcsize("@iiiiiiiIqfP12q") == ctypes.sizeof(RnRotaryDesc)
assert struct.calcsize("@10iIfqi15q") == ctypes.sizeof(RnLinearDesc)


def _bind(L):
    # descriptors as plain pointers: byref(...) of the structures above, or packed bytes
    for name, args, res in (
            ("rn_layernorm_forward", [_vp] * 8, _i32),
            ("rn_layernorm_backward_workspace_bytes", [_vp], _sz),
            ("rn_layernorm_backward", [_vp] * 9 + [_sz, _vp], _i32),
            ("rn_rmsnorm_forward", [_vp] * 8, _i32),
            ("rn_rmsnorm_backward_workspace_bytes", [_vp], _sz),
            ("rn_rmsnorm_backward", [_vp] * 8 + [_sz, _vp], _i32),
            ("rn_rotary", [_vp] * 7, _i32),
            ("rn_rotary_frequencies", [_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp, _vp], _i32),
            ("rn_linear_attention_workspace_bytes", [_vp], _sz),
            ("rn_linear_attention_chunked", [_vp] * 12 + [_sz, _vp], _i32),
            ("rn_linear_attention_step", [_vp] * 9, _i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res


_bind(lib)
_CODES = {torch.float32: RN_F32, torch.bfloat16: RN_BF16}


def _code(t: torch.dtype) -> int:
    c = _CODES.get(t)
    if c is None:
        raise TypeError(f"unsupported dtype {t}; use float32 or bfloat16")
    return c


# torch's own short ways to the current device and stream, where this torch has them
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(i, f, *args):
    """f(*args, stream) on the current stream of GPU i, which need not be the current GPU (a
    kernel launched on another device's stream would fail)."""
    if _current_device() == i:
        st = f(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            st = f(*args, _raw_stream(i))
    if st:
        _check(st)


def _device(first, *others) -> int:
    """The number of the GPU that all given tensors live on."""
    i = first.get_device()
    if i < 0:
        raise ValueError("tensors must live on the GPU")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError(f"tensors must be on one device ({first.device}); got {t.device}")
    return i


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _whole(t, dtype, shape, name):
    """A contiguous tensor of that type and shape, or None."""
    if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous {dtype} {tuple(shape)}; got {t.dtype} {tuple(t.shape)}")


def _get_workspace(workspace, need, like):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=like.device) if need else None
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    return workspace


# ---- layer norm ---------------------------------------------------------------------------

def _row_stride(t, name) -> int:
    """Elements between the rows of [..., d]: leading axes must step like one axis."""
    if t is None:
        return 0
    if t.is_contiguous():
        return t.shape[-1]
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    stride, span = None, 1
    for n, s in zip(t.shape[-2::-1], t.stride()[-2::-1]):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != stride * span:
            raise ValueError(f"{name}: the leading axes must have one common row stride")
        span *= n
    return t.shape[-1] if stride is None else stride


def _new(x, dtype):
    """A new contiguous tensor of x's shape."""
    if x.dtype == dtype and x.is_contiguous():
        return torch.empty_like(x)
    return x.new_empty(x.shape, dtype=dtype)


def _like(t, x, name):
    if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
        raise ValueError(f"{name} must be {x.dtype} {tuple(x.shape)}; got {t.dtype} {tuple(t.shape)}")


def rn_layernorm(x, weight=None, bias=None, eps=1e-5, *, residual=None, sum_out=None, out=None,
                 out_dtype=None):
    """Layer norm over the last axis of x [..., d], after adding ``residual`` (same shape and
    type) where given. weight, bias: float32 [d] or None. Returns out, or (out, sum) where a
    residual or ``sum_out`` is given; sum = x + residual in x's type (the next residual
    stream). ``sum_out`` and ``out`` (of x's type) may be x or residual, not both the same one."""
    dev = _device(x, residual, weight, bias, sum_out, out)
    shape = x.shape
    d = shape[-1] if shape else 0
    n = x.numel()
    if n == 0 or d == 0:
        raise ValueError(f"x must be [..., d] with at least one row; got {tuple(shape)}")
    _like(residual, x, "residual")
    _whole(weight, torch.float32, (d,), "weight")
    _whole(bias, torch.float32, (d,), "bias")
    if out is None:
        out = _new(x, x.dtype if out_dtype is None else out_dtype)
    elif out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out must be {out_dtype or out.dtype} {tuple(shape)}; got {out.dtype} {tuple(out.shape)}")
    if sum_out is None:
        if residual is not None:
            sum_out = _new(x, x.dtype)
    else:
        _like(sum_out, x, "sum_out")
    desc = _pack_norm(n // d, d, _code(x.dtype), _code(out.dtype), eps, _row_stride(x, "x"),
                      _row_stride(residual, "residual"), _row_stride(sum_out, "sum_out"), _row_stride(out, "out"))
    _call(dev, lib.rn_layernorm_forward, desc, x.data_ptr(), _p(residual), _p(weight), _p(bias), _p(sum_out),
          out.data_ptr())
    return out if sum_out is None else (out, sum_out)


def _norm_backward_desc(dout, x, eps, dsum, dx):
    d = x.shape[-1]
    return _pack_norm(x.numel() // d, d, _code(x.dtype), _code(dout.dtype), eps, _row_stride(x, "x"),
                      _row_stride(dsum, "dsum"), _row_stride(dx, "dx"), _row_stride(dout, "dout"))


def rn_layernorm_backward_workspace_bytes(dout, x) -> int:
    return int(lib.rn_layernorm_backward_workspace_bytes(_norm_backward_desc(dout, x, 0.0, None, x)))


def rn_layernorm_backward(dout, x, weight=None, eps=1e-5, *, dsum=None, dx=None, want_dweight=True,
                          want_dbias=True, workspace=None):
    """Gradients of ``rn_layernorm``: x are the rows it normalised (its sum where it had a
    residual), ``dsum`` the gradient that reaches this sum by its other path, in x's type.
    Returns a dict with dx (the gradient of x and of the residual; in x's type) and, unless not
    wanted, dweight and dbias (float32 [d]). ``dx`` may be x, dsum, or dout of x's type."""
    dev = _device(x, dout, weight, dsum, dx, workspace)
    if x.numel() == 0 or x.dim() == 0:
        raise ValueError(f"x must be [..., d] with at least one row; got {tuple(x.shape)}")
    d = x.shape[-1]
    if dout.shape != x.shape:
        raise ValueError(f"dout must have x's shape {tuple(x.shape)}; got {tuple(dout.shape)}")
    _whole(weight, torch.float32, (d,), "weight")
    _like(dsum, x, "dsum")
    if dx is None:
        dx = _new(x, x.dtype)
    else:
        _like(dx, x, "dx")
    desc = _norm_backward_desc(dout, x, eps, dsum, dx)
    got = {"dx": dx}
    if want_dweight:
        got["dweight"] = torch.empty(d, dtype=torch.float32, device=x.device)
    if want_dbias:
        got["dbias"] = torch.empty(d, dtype=torch.float32, device=x.device)
    if want_dweight or want_dbias:
        workspace = _get_workspace(workspace, lib.rn_layernorm_backward_workspace_bytes(desc), x)
    else:
        workspace = None
    _call(dev, lib.rn_layernorm_backward, desc, dout.data_ptr(), x.data_ptr(), _p(weight), _p(dsum), dx.data_ptr(),
          _p(got.get("dweight")), _p(got.get("dbias")), _p(workspace), 0 if workspace is None else workspace.numel())
    return got


# ---- root-mean-square norm ----------------------------------------------------------------

_HELD8 = {torch.float8_e4m3fn: RN_E4M3, torch.int8: RN_INT8}


def rn_rmsnorm(x, weight=None, eps=1e-5, *, residual=None, sum_out=None, out=None, out_dtype=None, group=0,
               scale_out=None):
    """Root-mean-square norm over the last axis of x [..., d], after adding ``residual`` (same shape
    and type) where given: y = h / sqrt(mean(h^2) + eps) * weight. weight: float32 [d] or None.

    ``out_dtype`` (default: x's type): float32, bfloat16, or torch.float8_e4m3fn / torch.int8 with a
    float32 scale for each row ([...]) or, with ``group`` 32, 64 or 128, for each so many columns
    ([..., ceil(d / group)]); out * scale stands for y. Returns out, and behind it the sum x + residual
    in x's type where a residual or ``sum_out`` is given, and the scale where out is of 8 bits.
    ``sum_out`` and ``out`` (of x's type) may be x or residual, not both the same one."""
    dev = _device(x, residual, weight, sum_out, out, scale_out)
    shape, kind = x.shape, x.dtype
    d = shape[-1] if shape else 0
    n = x.numel()
    if n == 0 or d == 0:
        raise ValueError(f"x must be [..., d] with at least one row; got {tuple(shape)}")
    if weight is not None:
        _whole(weight, torch.float32, (d,), "weight")
    xs = _row_stride(x, "x")
    rs = ss = os = d                      # new tensors are contiguous
    if residual is not None:
        _like(residual, x, "residual")
        rs = _row_stride(residual, "residual")
    if out is None:
        out = _new(x, kind if out_dtype is None else out_dtype)
    else:
        if out.shape != shape or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out must be {out_dtype or out.dtype} {tuple(shape)}; got {out.dtype} {tuple(out.shape)}")
        os = _row_stride(out, "out")
    if sum_out is not None:
        _like(sum_out, x, "sum_out")
        ss = _row_stride(sum_out, "sum_out")
    elif residual is not None:
        sum_out = _new(x, kind)
    code, scale, step = _HELD8.get(out.dtype), None, 0
    if code is None:
        code = _code(out.dtype)
        if scale_out is not None:
            raise ValueError("scale_out goes with an output of 8 bits")
    else:
        step = -(-d // group) if group > 0 else 1
        sizes = (*shape[:-1], step) if group else shape[:-1]
        if scale_out is None:
            scale = x.new_empty(sizes, dtype=torch.float32)
        else:
            _whole(scale_out, torch.float32, sizes, "scale_out")
            scale = scale_out
    _call(dev, lib.rn_rmsnorm_forward, _pack_rms(n // d, d, _code(kind), code, group, eps, xs, rs, ss, os, step), x.data_ptr(),
          _p(residual), _p(weight), _p(sum_out), out.data_ptr(), _p(scale))
    if scale is None:
        return out if sum_out is None else (out, sum_out)
    return (out, scale) if sum_out is None else (out, sum_out, scale)


def _rms_backward_desc(dout, x, eps, dsum, dx):
    d = x.shape[-1]
    return _pack_rms(x.numel() // d, d, _code(x.dtype), _code(dout.dtype), 0, eps, _row_stride(x, "x"),
                     _row_stride(dsum, "dsum"), _row_stride(dx, "dx"), _row_stride(dout, "dout"), 0)


def rn_rmsnorm_backward_workspace_bytes(dout, x) -> int:
    return int(lib.rn_rmsnorm_backward_workspace_bytes(_rms_backward_desc(dout, x, 0.0, None, x)))


def rn_rmsnorm_backward(dout, x, weight=None, eps=1e-5, *, dsum=None, dx=None, want_dweight=True, workspace=None):
    """Gradients of ``rn_rmsnorm``'s y: x are the rows it normalised (its sum where it had a residual),
    ``dsum`` the gradient that reaches this sum by its other path, in x's type. Returns a dict with dx
    (the gradient of x and of the residual; in x's type) and, unless not wanted, dweight (float32 [d]).
    ``dx`` may be x, dsum, or dout of x's type."""
    dev = _device(x, dout, weight, dsum, dx, workspace)
    if x.numel() == 0 or x.dim() == 0:
        raise ValueError(f"x must be [..., d] with at least one row; got {tuple(x.shape)}")
    d = x.shape[-1]
    if dout.shape != x.shape:
        raise ValueError(f"dout must have x's shape {tuple(x.shape)}; got {tuple(dout.shape)}")
    _whole(weight, torch.float32, (d,), "weight")
    _like(dsum, x, "dsum")
    if dx is None:
        dx = _new(x, x.dtype)
    else:
        _like(dx, x, "dx")
    desc = _rms_backward_desc(dout, x, eps, dsum, dx)
    got = {"dx": dx}
    if want_dweight:
        got["dweight"] = torch.empty(d, dtype=torch.float32, device=x.device)
        workspace = _get_workspace(workspace, lib.rn_rmsnorm_backward_workspace_bytes(desc), x)
    else:
        workspace = None
    _call(dev, lib.rn_rmsnorm_backward, desc, dout.data_ptr(), x.data_ptr(), _p(weight), _p(dsum), dx.data_ptr(),
          _p(got.get("dweight")), _p(workspace), 0 if workspace is None else workspace.numel())
    return got


# ---- rotary positions -----------------------------------------------------------------------

def _bhn(t, name):
    """Strides of [B, H, N, d] with a contiguous last axis."""
    st = t.stride()
    if st[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return st[:3]


def _new_like(t, shape, dtype):
    """A new tensor of the given shape [B, H, N, d], token-major in memory where t is."""
    if t.dtype == dtype and t.shape == shape:
        return torch.empty_like(t)
    B, H, N, d = shape
    _, h, n, _ = t.stride()
    if h < n:                             # [B, N, H, d] in memory
        return torch.empty_strided((B, H, N, d), (N * H * d, d, H * d, 1), dtype=dtype, device=t.device)
    return torch.empty((B, H, N, d), dtype=dtype, device=t.device)


_NO_STRIDE = (0, 0, 0)


def rn_rotary(q, k=None, theta=None, *, pos0=0, pos=None, half=False, inverse=False, magnitude=1.0,
              q_out=None, k_out=None):
    """Rotary positions on q [B, H_q, N, d] and k [B, H_k, N, d] (k may be None): pair j of the
    first 2 len(theta) coordinates of every head is turned by position * theta[j] and scaled by
    ``magnitude``; the others are copied. Pairs are (2j, 2j+1), or (j, j + len(theta)) with
    ``half``. ``inverse`` turns back: the transpose, so it takes output gradients to input
    gradients. theta: host angles (float64 is kept). pos: device int64 [B] (positions of the
    first tokens) or [B, N]; None = ``pos0`` + token. Returns q_out, or (q_out, k_out); an output
    given may be its input (in place)."""
    if theta is None:
        raise ValueError("theta is required")
    dev = _device(q, k, pos, q_out, k_out)
    sq, sk = q.shape, None if k is None else k.shape
    if len(sq) != 4 or (k is not None and (len(sk) != 4 or k.dtype != q.dtype or sk[0] != sq[0] or sk[2] != sq[2] or
                                           sk[3] != sq[3])):
        raise ValueError(f"expected q [B,H_q,N,d] and k [B,H_k,N,d] of one type; got {q.dtype} {tuple(q.shape)}"
                         + ("" if k is None else f", {k.dtype} {tuple(k.shape)}"))
    if 0 in sq or (k is not None and 0 in sk):
        raise ValueError("q and k must not be empty")
    B, Hq, N, d = sq
    th = np.ascontiguousarray(theta, dtype=np.float64)
    if th.ndim != 1:
        raise ValueError("theta must be one-dimensional")
    flags = (RN_ROTARY_HALF if half else 0) | (RN_ROTARY_INVERSE if inverse else 0)
    if pos is not None:
        if pos.dtype != torch.int64 or not pos.is_contiguous() or pos.shape not in ((B,), (B, N)):
            raise ValueError(f"pos must be contiguous int64 [{B}] or [{B}, {N}]; got {pos.dtype} {tuple(pos.shape)}")
        if pos.dim() == 2:
            flags |= RN_ROTARY_POS_TOKEN
    for t, like, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if t is not None:
            if like is None:
                raise ValueError("k_out without k")
            _like(t, like, name)
    if q_out is None:
        q_out = torch.empty_like(q)         # dense, its axes in memory as q's
    if k is not None and k_out is None:
        k_out = torch.empty_like(k)
    qs, qos = _bhn(q, "q"), _bhn(q_out, "q_out")
    ks, kos = (_NO_STRIDE, _NO_STRIDE) if k is None else (_bhn(k, "k"), _bhn(k_out, "k_out"))
    desc = _pack_rotary(B, N, Hq, 0 if k is None else sk[1], d, 2 * len(th), _code(q.dtype), flags, pos0,
                        magnitude, th.ctypes.data, *qs, *ks, *qos, *kos)
    _call(dev, lib.rn_rotary, desc, _p(pos), q.data_ptr(), _p(k), q_out.data_ptr(), _p(k_out))
    return q_out if k is None else (q_out, k_out)


_ROPE_KINDS = {"plain": RN_ROPE_PLAIN, "linear": RN_ROPE_LINEAR, "base": RN_ROPE_BASE, "by_parts": RN_ROPE_BY_PARTS}


def rn_rotary_frequencies(rot, base=10000.0, kind="plain", *, factor=1.0, length=4096.0, slow=1.0, fast=32.0):
    """Angles of rot/2 coordinate pairs (float64 host array) and the magnitude to pass with
    them. kind: "plain", or stretched for contexts ``factor`` times the trained ``length``:
    "linear" (every angle / factor), "base" (a larger base), "by_parts" (pairs turning at most
    ``slow`` times over the trained length / factor, those turning ``fast`` times unchanged,
    mixed between)."""
    if kind not in _ROPE_KINDS:
        raise ValueError(f"kind must be one of {', '.join(_ROPE_KINDS)}; got {kind!r}")
    theta = np.empty(max(int(rot) // 2, 1), dtype=np.float64)
    m = _f32()
    _check(lib.rn_rotary_frequencies(rot, base, _ROPE_KINDS[kind], factor, length, slow, fast, theta.ctypes.data,
                                     ctypes.addressof(m)))
    return theta, m.value


# ---- linear attention -----------------------------------------------------------------------

def _linear_shapes(q, k, v, g):
    sq, sk, sv, sg = q.shape, k.shape, v.shape, g.shape
    if not (len(sq) == len(sk) == len(sv) == 4):
        raise ValueError(f"expected q [B,H_q,N,d_k], k [B,H_k,N,d_k], v [B,H_v,N,d_v]; got {tuple(sq)}, {tuple(sk)}, "
                         f"{tuple(sv)}")
    B, _, rows, dk = sq
    if sk[0] != B or sk[2] != rows or sk[3] != dk or sv[0] != B or sv[2] != rows:
        raise ValueError(f"q, k and v must agree in batch and tokens, q and k in d_k; got {tuple(sq)}, {tuple(sk)}, "
                         f"{tuple(sv)}")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    if len(sg) != 3 or g.dtype != torch.float32 or sg[0] != B or sg[2] != rows:
        raise ValueError(f"log_decay must be float32 [{B}, H, {rows}]; got {g.dtype} {tuple(sg)}")


def _linear_desc(q, k, v, g, S, N, T, n_slots, out_dtype, flags, qk_scale, out):
    return _pack_linear(S, N, g.shape[1], q.shape[1], k.shape[1], v.shape[1], q.shape[3], v.shape[3], _code(q.dtype),
                        _code(out_dtype), flags, qk_scale, T, n_slots, *_bhn(q, "q"), *_bhn(k, "k"), *_bhn(v, "v"),
                        *g.stride(), *out)


def _linear_out(out, q, v, H, out_dtype):
    """The output and whether it is new."""
    shape = (v.shape[0], H, v.shape[2], v.shape[3])
    od = (q.dtype if out is None else out.dtype) if out_dtype is None else out_dtype
    if out is None:
        return _new_like(v, shape, od), True
    if out.shape != shape or out.dtype != od:
        raise ValueError(f"out must be {od} {shape}; got {out.dtype} {tuple(out.shape)}")
    return out, False


def _int32(t, n, name):
    if t is not None and (t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous int32 [{n}]; got {t.dtype} {tuple(t.shape)}")


def _linear_state(s, shape, slots, name):
    if s is None:
        return
    if s.dtype != torch.float32 or not s.is_contiguous() or s.dim() != 4 or s.shape[1:] != shape[1:] or \
            (slots is None and s.shape[0] != shape[0]) or s.shape[0] < 1:
        raise ValueError(f"{name} must be contiguous float32 [{'slots' if slots is not None else shape[0]}, "
                         f"{shape[1]}, {shape[2]}, {shape[3]}]; got {s.dtype} {tuple(s.shape)}")


def _linear_call(q, k, v, g, qk_scale, lengths, cu, max_len, state_in, state_out, slots, out, out_dtype, generic):
    B, rows = q.shape[0], q.shape[2]
    if cu is not None:
        if B != 1 or lengths is not None or cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("a packed batch is [1, H, T, d] with cu_seqlens [S + 1] and without lengths")
        S, T, N = cu.numel() - 1, rows, rows
    else:
        S, T, N = B, 0, rows
    if max_len is not None:
        if not 1 <= max_len <= N:
            raise ValueError(f"max_len={max_len} outside [1, {N}]")
        N = max_len
    flags = RN_LINEAR_GENERIC if generic else 0
    H = g.shape[1]
    out, new = _linear_out(out, q, v, H, out_dtype)
    if new and (cu is not None or lengths is not None):
        flags |= RN_LINEAR_ZERO_REST
    if new and cu is None and N < rows:
        out[:, :, N:].zero_()
    shape = (S, H, q.shape[-1], v.shape[-1])
    if slots is not None and state_out is True:
        raise ValueError("with slots, state_out must be a tensor")
    _linear_state(state_in, shape, slots, "state_in")
    if state_out is True:
        state_out = torch.empty(shape, dtype=torch.float32, device=q.device)
    elif state_out is False:
        state_out = None
    else:
        _linear_state(state_out, shape, slots, "state_out")
    n_slots = 0
    if slots is not None:
        sizes = {s.shape[0] for s in (state_in, state_out) if s is not None}
        if len(sizes) > 1:
            raise ValueError("state_in and state_out must have the same number of slots")
        n_slots = sizes.pop() if sizes else 1
    desc = _linear_desc(q, k, v, g, S, N, T, n_slots, out.dtype, flags, qk_scale, _bhn(out, "out"))
    return desc, S, out, state_out


def rn_linear_attention_workspace_bytes(q, k, v, log_decay, *, cu_seqlens=None, max_len=None, out=None,
                                        out_dtype=None, force_generic=False) -> int:
    """Bytes of workspace ``rn_linear_attention_chunked`` needs for these tensors (and the ``out``
    it is given, where it is)."""
    _linear_shapes(q, k, v, log_decay)
    B, rows = q.shape[0], q.shape[2]
    S, T = (B, 0) if cu_seqlens is None else (cu_seqlens.numel() - 1, rows)
    if out is None:
        o = (log_decay.shape[1] * rows * v.shape[-1], rows * v.shape[-1], v.shape[-1])
        dtype = out_dtype or q.dtype
    else:
        o, dtype = _bhn(out, "out"), out.dtype
    desc = _linear_desc(q, k, v, log_decay, S, max_len or rows, T, 0, dtype,
                        RN_LINEAR_GENERIC if force_generic else 0, 1.0, o)
    return int(lib.rn_linear_attention_workspace_bytes(desc))


def rn_linear_attention_chunked(q, k, v, log_decay, *, qk_scale=1.0, lengths=None, cu_seqlens=None, max_len=None,
                                state_in=None, state_out=None, slots=None, out=None, out_dtype=None,
                                workspace=None, force_generic=False):
    """Linear attention with a decay per head and token over prompts:
    S_t = exp(g_t) S_{t-1} + k_t^T v_t, o_t = qk_scale q_t S_t; returns (out, state_out).

    q [B, H_q, N, d_k], k [B, H_k, N, d_k], v [B, H_v, N, d_v]; log_decay float32 [B, H, N]
    (<= 0; -inf clears the state; a stride of 0 along N gives one decay per head). H_q, H_k and
    H_v divide H. Padded batch: ``lengths`` device int32 [B] or None. Packed batch: B = 1 and
    ``cu_seqlens`` device int32 [S + 1], first entry 0. ``max_len``: no sequence is longer (host
    number; longer ones are cut); many short packed sequences run best with it. Rows of no sequence are not written (zero in a new out).
    state_in, state_out: float32 [S, H, d_k, d_v], or pools [slots, H, d_k, d_v] with ``slots``
    device int32 [S] (distinct; -1: start from zeros, keep nothing); state_out may be True (new;
    not with slots), None/False (discarded) or state_in itself."""
    dev = _device(q, k, v, log_decay, lengths, cu_seqlens, slots, out, workspace, state_in,
                  state_out if isinstance(state_out, torch.Tensor) else None)
    _linear_shapes(q, k, v, log_decay)
    desc, S, out, state_out = _linear_call(q, k, v, log_decay, qk_scale, lengths, cu_seqlens, max_len, state_in,
                                           state_out, slots, out, out_dtype, force_generic)
    _int32(lengths, S, "lengths")
    _int32(cu_seqlens, S + 1, "cu_seqlens")
    _int32(slots, S, "slots")
    workspace = _get_workspace(workspace, lib.rn_linear_attention_workspace_bytes(desc), q)
    _call(dev, lib.rn_linear_attention_chunked, desc, _p(cu_seqlens), _p(lengths), _p(slots), q.data_ptr(),
          k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(state_in), _p(state_out), out.data_ptr(), _p(workspace),
          0 if workspace is None else workspace.numel())
    return out, state_out


def rn_linear_attention_step(q, k, v, log_decay, state, *, qk_scale=1.0, slots=None, out=None, out_dtype=None):
    """One token for each of S sequences: q [S, H_q, 1, d_k], k, v, log_decay [S, H, 1] as in
    ``rn_linear_attention_chunked``; ``state`` (float32 [S, H, d_k, d_v], or a pool with ``slots``)
    is updated in place. Returns out [S, H, 1, d_v]; a sequence with slot -1 is skipped, its row
    of out set to zero."""
    dev = _device(q, k, v, log_decay, state, slots, out)
    _linear_shapes(q, k, v, log_decay)
    if q.shape[2] != 1:
        raise ValueError(f"the step takes one token a sequence: q [S,H_q,1,d_k]; got {tuple(q.shape)}")
    S, H = q.shape[0], log_decay.shape[1]
    out, _ = _linear_out(out, q, v, H, out_dtype)
    _linear_state(state, (S, H, q.shape[-1], v.shape[-1]), slots, "state")
    _int32(slots, S, "slots")
    desc = _linear_desc(q, k, v, log_decay, S, 1, 0, state.shape[0], out.dtype, 0, qk_scale, _bhn(out, "out"))
    _call(dev, lib.rn_linear_attention_step, desc, _p(slots), q.data_ptr(), k.data_ptr(), v.data_ptr(),
          log_decay.data_ptr(), state.data_ptr(), out.data_ptr())
    return out
