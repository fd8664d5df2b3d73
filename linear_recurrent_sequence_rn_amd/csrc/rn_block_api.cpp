// C ABI of the operators around retention (layer norm, rotary positions, linear attention):
// host-side validation and dispatch, before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <utility>

#include "rn_kernels.h"
#include "rn_retention.h"

namespace {

using rn::fail;
using rn::hip_status;

bool dtype_ok(rn_dtype d) { return d == RN_F32 || d == RN_BF16; }
int64_t size_of(rn_dtype d) { return d == RN_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int kMaxNorm = 16384;

rn_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return RN_OK;
  if (!ws || have < need)
    return fail(RN_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws ? have : size_t(0), need);
  if (!aligned(ws, 256)) return fail(RN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return RN_OK;
}

// ---- layer norm ---------------------------------------------------------------------------

rn_status check_norm(const rn_norm_desc* d, rn::NormCall* n) {
  if (!d) return fail(RN_ERR_INVALID_ARG, "desc is NULL");
  if (d->rows < 1 || d->d < 1)
    return fail(RN_ERR_INVALID_ARG, "sizes must be >= 1 (rows=%lld d=%d)", (long long)d->rows, d->d);
  if (d->rows > (int64_t(1) << 40)) return fail(RN_ERR_UNSUPPORTED, "rows=%lld > 2^40", (long long)d->rows);
  if (d->d > kMaxNorm) return fail(RN_ERR_UNSUPPORTED, "d=%d > %d", d->d, kMaxNorm);
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype))
    return fail(RN_ERR_INVALID_ARG, "unknown dtype (in=%d out=%d)", d->in_dtype, d->out_dtype);
  if (!(d->eps >= 0.f && std::isfinite(d->eps))) return fail(RN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  for (int64_t s : {d->x_stride, d->res_stride, d->sum_stride, d->out_stride})
    if (s < 0 || s > kMaxStride) return fail(RN_ERR_INVALID_ARG, "row stride %lld outside [0, 2^40]", (long long)s);
  std::memset(n, 0, sizeof(*n));
  n->rows = d->rows; n->d = d->d; n->in_dt = d->in_dtype; n->out_dt = d->out_dtype; n->eps = d->eps;
  n->xs = d->x_stride; n->rs = d->res_stride; n->ss = d->sum_stride; n->os = d->out_stride;
  return RN_OK;
}

// 16-byte vectors of the input type: every row of every tensor starts and ends on one.
bool norm_vectors(const rn::NormCall& n) {
  const int v = n.in_dt == RN_BF16 ? 8 : 4;
  auto ok = [&](const void* p, int64_t stride) { return !p || (aligned(p, 16) && (n.rows == 1 || stride % v == 0)); };
  // (an f32 out beside a bf16 input has its rows on 32 bytes, a bf16 out beside f32 on 8)
  return n.d % v == 0 && ok(n.x, n.xs) && ok(n.r, n.rs) && ok(n.sum, n.ss) && ok(n.out, n.os) && ok(n.dout, n.os) &&
         ok(n.w, 0) && ok(n.b, 0);
}

rn_status check_rows_out(const rn::NormCall& n, int64_t stride, const char* what) {
  if (n.rows > 1 && stride < n.d)
    return fail(RN_ERR_INVALID_ARG, "%s: row stride %lld < d=%d (its rows would overlap)", what, (long long)stride, n.d);
  return RN_OK;
}

rn_status check_elements(const void* p, rn_dtype dt, const char* what) {
  if (!aligned(p, size_of(dt)))
    return fail(RN_ERR_INVALID_ARG, "%s must be %d-byte aligned", what, int(size_of(dt)));
  return RN_OK;
}

// ---- rotary -------------------------------------------------------------------------------

rn_status check_strides(const int64_t* s, const char* what) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > kMaxStride)
      return fail(RN_ERR_INVALID_ARG, "%s stride %lld outside [0, 2^40]", what, (long long)s[i]);
  return RN_OK;
}

// An output's elements must be distinct: ordered by stride, each axis has to step over all
// that the axes inside it cover.
rn_status check_distinct(const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int64_t d, const char* what) {
  int64_t st[3] = {s[0], s[1], s[2]}, n[3] = {n0, n1, n2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) { std::swap(st[i], st[j]); std::swap(n[i], n[j]); }
  __int128 span = d;   // stride * size may pass 64 bits
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < span)
      return fail(RN_ERR_INVALID_ARG, "%s: strides %lld, %lld, %lld make it overlap itself", what,
                  (long long)s[0], (long long)s[1], (long long)s[2]);
    span += static_cast<__int128>(st[i]) * (n[i] - 1);
  }
  return RN_OK;
}

// A tensor: three strided axes of elements of `es` bytes, and d contiguous ones.
struct Box {
  const void* p;
  int64_t es, s[3], n[3], d;
};

// Whether elements at i . s + [0, a.d) and diff + j . s + [0, b.d) meet, i and j inside the boxes: the
// steps k = i - j along the axes from `axis` on, ordered by falling stride, that bring diff near 0.
bool meets(int64_t diff, const Box& a, const Box& b, const int64_t* s, const int* order, int axis) {
  if (axis == 3) return diff < a.d * a.es && -diff < b.d * b.es;
  const int x = order[axis];
  const int64_t st = s[x] * a.es, up = a.n[x] - 1, down = b.n[x] - 1;
  if (st == 0) return meets(diff, a, b, s, order, axis + 1);
  const int64_t k0 = diff / st;           // (k st is at most st from diff, an address, away)
  for (int64_t k = k0 - 1; k <= k0 + 1; ++k)
    if (k <= up && -k <= down && meets(diff - k * st, a, b, s, order, axis + 1)) return true;
  return false;
}

// Whether an output overlaps another operand, as far as two tensors of one type and the same strides
// show it (of others nothing is said). The same tensor in both places is no overlap here.
bool overlaps(const Box& out, const Box& in) {
  if (!in.p || in.p == out.p || out.es != in.es) return false;
  int64_t s[3];
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i) {
    if (out.n[i] > 1 && in.n[i] > 1 && out.s[i] != in.s[i]) return false;
    s[i] = out.n[i] > 1 ? out.s[i] : in.n[i] > 1 ? in.s[i] : 0;
  }
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[order[j]] > s[order[i]]) std::swap(order[i], order[j]);
  const int64_t diff = static_cast<int64_t>(reinterpret_cast<uintptr_t>(in.p) - reinterpret_cast<uintptr_t>(out.p));
  return meets(diff, out, in, s, order, 0);
}

rn_status check_no_overlap(const Box& out, const Box& in, const char* what, const char* other) {
  if (overlaps(out, in)) return fail(RN_ERR_INVALID_ARG, "%s overlaps %s", what, other);
  return RN_OK;
}
Box box(const void* p, rn_dtype dt, const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int64_t d) {
  return Box{p, size_of(dt), {s[0], s[1], s[2]}, {n0, n1, n2}, d};
}
Box row_box(const void* p, rn_dtype dt, int64_t stride, const rn::NormCall& n) {
  return Box{p, size_of(dt), {0, 0, stride}, {1, 1, n.rows}, n.d};
}

// ---- linear attention -----------------------------------------------------------------------

rn_status check_linear(const rn_linear_desc* d, bool step, rn::LinCall* c) {
  if (!d) return fail(RN_ERR_INVALID_ARG, "desc is NULL");
  if (d->S < 1 || d->N < 1 || d->H < 1 || d->H_q < 1 || d->H_k < 1 || d->H_v < 1 || d->d_k < 1 || d->d_v < 1)
    return fail(RN_ERR_INVALID_ARG, "sizes must be >= 1 (S=%d N=%d H=%d H_q=%d H_k=%d H_v=%d d_k=%d d_v=%d)",
                d->S, d->N, d->H, d->H_q, d->H_k, d->H_v, d->d_k, d->d_v);
  if (d->H % d->H_q || d->H % d->H_k || d->H % d->H_v)
    return fail(RN_ERR_INVALID_ARG, "H_q=%d, H_k=%d and H_v=%d must divide H=%d", d->H_q, d->H_k, d->H_v, d->H);
  if (d->d_k > rn::kMaxDk) return fail(RN_ERR_UNSUPPORTED, "d_k=%d > %d", d->d_k, rn::kMaxDk);
  if (d->d_v > rn::kMaxDv) return fail(RN_ERR_UNSUPPORTED, "d_v=%d > %d", d->d_v, rn::kMaxDv);
  if (d->S > 65534) return fail(RN_ERR_UNSUPPORTED, "S=%d > 65534", d->S);
  if (d->H > 65535) return fail(RN_ERR_UNSUPPORTED, "H=%d > 65535", d->H);
  if (d->N > (1 << 30)) return fail(RN_ERR_UNSUPPORTED, "N=%d > 2^30", d->N);
  if (step && d->N != 1) return fail(RN_ERR_INVALID_ARG, "the step needs N == 1 (got %d)", d->N);
  if (!dtype_ok(d->in_dtype) || !dtype_ok(d->out_dtype))
    return fail(RN_ERR_INVALID_ARG, "unknown dtype (in=%d out=%d)", d->in_dtype, d->out_dtype);
  if (d->flags & ~(RN_LINEAR_ZERO_REST | RN_LINEAR_GENERIC))
    return fail(RN_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags);
  if (!std::isfinite(d->qk_scale)) return fail(RN_ERR_INVALID_ARG, "qk_scale is not finite");
  if (d->T < 0 || d->T > INT32_MAX) return fail(RN_ERR_INVALID_ARG, "T=%lld outside [0, 2^31 - 1]", (long long)d->T);
  if (step && d->T) return fail(RN_ERR_INVALID_ARG, "the step takes no packed batch (T=%lld)", (long long)d->T);
  if (d->T && d->N > d->T) return fail(RN_ERR_INVALID_ARG, "N=%d > T=%lld", d->N, (long long)d->T);
  rn_status s;
  if ((s = check_strides(d->q_stride, "q")) || (s = check_strides(d->k_stride, "k")) ||
      (s = check_strides(d->v_stride, "v")) || (s = check_strides(d->g_stride, "log_decay")) ||
      (s = check_strides(d->out_stride, "out")) ||
      (s = check_distinct(d->out_stride, d->T ? 1 : d->S, d->H, d->T ? d->T : d->N, d->d_v, "out")))
    return s;
  std::memset(c, 0, sizeof(*c));
  c->S = d->S; c->N = d->N; c->H = d->H; c->Hq = d->H_q; c->Hk = d->H_k; c->Hv = d->H_v;
  c->dk = d->d_k; c->dv = d->d_v;
  c->in_dt = d->in_dtype; c->out_dt = d->out_dtype;
  c->generic = d->flags & RN_LINEAR_GENERIC;
  c->zero_rest = d->flags & RN_LINEAR_ZERO_REST;
  c->scale = d->qk_scale;
  c->T = d->T; c->n_slots = d->n_slots;
  c->qs = d->q_stride; c->ks = d->k_stride; c->vs = d->v_stride; c->gs = d->g_stride; c->os = d->out_stride;
  return RN_OK;
}

rn_status check_linear_ptrs(const rn_linear_desc* d, const int32_t* slots, const void* q, const void* k, const void* v,
                            const float* g, const void* out, rn::LinCall* c) {
  if (!q || !k || !v || !g || !out) return fail(RN_ERR_INVALID_ARG, "q/k/v/log_decay/out pointer is NULL");
  if (!aligned(slots, 4)) return fail(RN_ERR_INVALID_ARG, "slots must be 4-byte aligned");
  if (slots && d->n_slots < 1) return fail(RN_ERR_INVALID_ARG, "n_slots=%d must be >= 1", d->n_slots);
  rn_status s;
  if ((s = check_elements(q, d->in_dtype, "q")) || (s = check_elements(k, d->in_dtype, "k")) ||
      (s = check_elements(v, d->in_dtype, "v")) || (s = check_elements(g, RN_F32, "log_decay")) ||
      (s = check_elements(out, d->out_dtype, "out")))
    return s;
  c->slots = slots; c->q = q; c->k = k; c->v = v; c->g = g; c->out = const_cast<void*>(out);
  return RN_OK;
}

// Blocks read q, k and v while others write out.
rn_status check_apart(const rn_linear_desc* d, const rn::LinCall& c) {
  if (c.out == c.q || c.out == c.k || c.out == c.v) return fail(RN_ERR_INVALID_ARG, "out must not be q, k or v");
  const int64_t S = d->T ? 1 : d->S, N = d->T ? d->T : d->N;
  const Box out = box(c.out, d->out_dtype, d->out_stride, S, d->H, N, d->d_v);
  rn_status s;
  if ((s = check_no_overlap(out, box(c.q, d->in_dtype, d->q_stride, S, d->H_q, N, d->d_k), "out", "q")) ||
      (s = check_no_overlap(out, box(c.k, d->in_dtype, d->k_stride, S, d->H_k, N, d->d_k), "out", "k")) ||
      (s = check_no_overlap(out, box(c.v, d->in_dtype, d->v_stride, S, d->H_v, N, d->d_v), "out", "v")))
    return s;
  return RN_OK;
}

}  // namespace

extern "C" {

rn_status rn_layernorm_forward(const rn_norm_desc* desc, const void* x, const void* residual, const float* weight,
                               const float* bias, void* sum_out, void* out, void* stream) {
  rn::NormCall n;
  rn_status s = check_norm(desc, &n);
  if (s != RN_OK) return s;
  if (!x || !out) return fail(RN_ERR_INVALID_ARG, "x/out pointer is NULL");
  if ((s = check_elements(x, desc->in_dtype, "x")) || (s = check_elements(residual, desc->in_dtype, "residual")) ||
      (s = check_elements(sum_out, desc->in_dtype, "sum_out")) || (s = check_elements(out, desc->out_dtype, "out")) ||
      (s = check_elements(weight, RN_F32, "weight")) || (s = check_elements(bias, RN_F32, "bias")) ||
      (s = check_rows_out(n, n.os, "out")) || (sum_out && (s = check_rows_out(n, n.ss, "sum_out"))))
    return s;
  if (out == sum_out) return fail(RN_ERR_INVALID_ARG, "out and sum_out must differ");
  if ((out == x && (desc->in_dtype != desc->out_dtype || n.os != n.xs)) ||
      (out == residual && (desc->in_dtype != desc->out_dtype || n.os != n.rs)) ||
      (sum_out && ((sum_out == x && n.ss != n.xs) || (sum_out == residual && n.ss != n.rs))))
    return fail(RN_ERR_INVALID_ARG, "in place needs equal types and strides");
  const Box bx = row_box(x, desc->in_dtype, n.xs, n), br = row_box(residual, desc->in_dtype, n.rs, n),
            bs = row_box(sum_out, desc->in_dtype, n.ss, n), bo = row_box(out, desc->out_dtype, n.os, n);
  if ((s = check_no_overlap(bo, bx, "out", "x")) || (s = check_no_overlap(bo, br, "out", "residual")) ||
      (s = check_no_overlap(bo, bs, "out", "sum_out")) ||
      (sum_out && ((s = check_no_overlap(bs, bx, "sum_out", "x")) || (s = check_no_overlap(bs, br, "sum_out", "residual")))))
    return s;
  n.x = x; n.r = residual; n.w = weight; n.b = bias; n.sum = sum_out; n.out = out;
  n.vec = norm_vectors(n);
  rn::clear_error();
  return hip_status(rn::launch_layernorm(n, static_cast<hipStream_t>(stream)), "layer norm launch");
}

size_t rn_layernorm_backward_workspace_bytes(const rn_norm_desc* desc) {
  rn::NormCall n;
  if (check_norm(desc, &n) != RN_OK) return 0;
  return (rn::norm_backward_ws_bytes(n) + 255) & ~size_t(255);
}

rn_status rn_layernorm_backward(const rn_norm_desc* desc, const void* dout, const void* x, const float* weight,
                                const void* dsum, void* dx, float* dweight, float* dbias, void* workspace,
                                size_t workspace_bytes, void* stream) {
  rn::NormCall n;
  rn_status s = check_norm(desc, &n);
  if (s != RN_OK) return s;
  if (!dout || !x || !dx) return fail(RN_ERR_INVALID_ARG, "dout/x/dx pointer is NULL");
  if ((s = check_elements(x, desc->in_dtype, "x")) || (s = check_elements(dsum, desc->in_dtype, "dsum")) ||
      (s = check_elements(dx, desc->in_dtype, "dx")) || (s = check_elements(dout, desc->out_dtype, "dout")) ||
      (s = check_elements(weight, RN_F32, "weight")) || (s = check_elements(dweight, RN_F32, "dweight")) ||
      (s = check_elements(dbias, RN_F32, "dbias")) || (s = check_rows_out(n, n.ss, "dx")))
    return s;
  if ((dx == dout && (desc->in_dtype != desc->out_dtype || n.ss != n.os)) || (dx == x && n.ss != n.xs) ||
      (dx == dsum && n.ss != n.rs))
    return fail(RN_ERR_INVALID_ARG, "in place needs equal types and strides");
  const Box bd = row_box(dx, desc->in_dtype, n.ss, n);
  if ((s = check_no_overlap(bd, row_box(x, desc->in_dtype, n.xs, n), "dx", "x")) ||
      (s = check_no_overlap(bd, row_box(dout, desc->out_dtype, n.os, n), "dx", "dout")) ||
      (s = check_no_overlap(bd, row_box(dsum, desc->in_dtype, n.rs, n), "dx", "dsum")))
    return s;
  if (dweight || dbias) {
    const size_t need = (rn::norm_backward_ws_bytes(n) + 255) & ~size_t(255);
    if ((s = check_workspace(workspace, workspace_bytes, need)) != RN_OK) return s;
  }
  n.backward = true;
  n.x = x; n.r = dsum; n.w = weight; n.sum = dx; n.dout = dout; n.dw = dweight; n.db = dbias; n.ws = workspace;
  n.vec = norm_vectors(n);
  rn::clear_error();
  return hip_status(rn::launch_layernorm(n, static_cast<hipStream_t>(stream)), "layer norm backward launch");
}

rn_status rn_rotary(const rn_rotary_desc* desc, const int64_t* pos, const void* q, const void* k, void* q_out,
                    void* k_out, void* stream) {
  const rn_rotary_desc* d = desc;
  if (!d) return fail(RN_ERR_INVALID_ARG, "desc is NULL");
  if (d->B < 1 || d->N < 1 || d->H_q < 1 || d->H_k < 0 || d->d < 2)
    return fail(RN_ERR_INVALID_ARG, "sizes out of range (B=%d N=%d H_q=%d H_k=%d d=%d)", d->B, d->N, d->H_q, d->H_k, d->d);
  if (d->rot < 2 || d->rot % 2 || d->rot > d->d)
    return fail(RN_ERR_INVALID_ARG, "rot=%d must be even, in [2, d=%d]", d->rot, d->d);
  if (d->rot > rn::kMaxRot) return fail(RN_ERR_UNSUPPORTED, "rot=%d > %d", d->rot, rn::kMaxRot);
  if (d->d > rn::kMaxDv) return fail(RN_ERR_UNSUPPORTED, "d=%d > %d", d->d, rn::kMaxDv);
  if (int64_t(d->H_q) + d->H_k > 65535) return fail(RN_ERR_UNSUPPORTED, "H_q + H_k = %lld > 65535", (long long)d->H_q + d->H_k);
  if (int64_t(d->B) * d->N > INT32_MAX)
    return fail(RN_ERR_UNSUPPORTED, "B*N=%lld > 2^31 - 1", (long long)d->B * d->N);
  if (!dtype_ok(d->dtype)) return fail(RN_ERR_INVALID_ARG, "unknown dtype (%d)", d->dtype);
  if (d->flags & ~(RN_ROTARY_HALF | RN_ROTARY_INVERSE | RN_ROTARY_POS_TOKEN))
    return fail(RN_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags);
  if (d->pos0 < 0 || d->pos0 > (int64_t(1) << 40))
    return fail(RN_ERR_INVALID_ARG, "pos0=%lld outside [0, 2^40]", (long long)d->pos0);
  if (!std::isfinite(d->magnitude)) return fail(RN_ERR_INVALID_ARG, "magnitude is not finite");
  if (!d->theta) return fail(RN_ERR_INVALID_ARG, "theta is NULL");
  for (int j = 0; j < d->rot / 2; ++j)
    if (!std::isfinite(d->theta[j])) return fail(RN_ERR_INVALID_ARG, "theta[%d] is not finite", j);
  if ((d->flags & RN_ROTARY_POS_TOKEN) && !pos) return fail(RN_ERR_INVALID_ARG, "RN_ROTARY_POS_TOKEN needs pos");
  if (!aligned(pos, 8)) return fail(RN_ERR_INVALID_ARG, "pos must be 8-byte aligned");
  if (!q || !q_out || (d->H_k && (!k || !k_out))) return fail(RN_ERR_INVALID_ARG, "q/k/q_out/k_out pointer is NULL");
  rn_status s;
  if ((s = check_strides(d->q_stride, "q")) || (s = check_strides(d->q_out_stride, "q_out")) ||
      (s = check_elements(q, d->dtype, "q")) || (s = check_elements(q_out, d->dtype, "q_out")) ||
      (s = check_distinct(d->q_out_stride, d->B, d->H_q, d->N, d->d, "q_out")))
    return s;
  if (q == q_out && std::memcmp(d->q_stride, d->q_out_stride, sizeof(d->q_stride)))
    return fail(RN_ERR_INVALID_ARG, "q in place needs equal strides");
  if (d->H_k) {
    if ((s = check_strides(d->k_stride, "k")) || (s = check_strides(d->k_out_stride, "k_out")) ||
        (s = check_elements(k, d->dtype, "k")) || (s = check_elements(k_out, d->dtype, "k_out")) ||
        (s = check_distinct(d->k_out_stride, d->B, d->H_k, d->N, d->d, "k_out")))
      return s;
    if (k == k_out && std::memcmp(d->k_stride, d->k_out_stride, sizeof(d->k_stride)))
      return fail(RN_ERR_INVALID_ARG, "k in place needs equal strides");
    if (q_out == k_out) return fail(RN_ERR_INVALID_ARG, "q_out and k_out must differ");
    if (q_out == k || k_out == q) return fail(RN_ERR_INVALID_ARG, "an output may only be its own input");
  }
  const Box bq = box(q, d->dtype, d->q_stride, d->B, d->H_q, d->N, d->d), bqo = box(q_out, d->dtype, d->q_out_stride, d->B, d->H_q, d->N, d->d);
  if ((s = check_no_overlap(bqo, bq, "q_out", "q"))) return s;
  if (d->H_k) {
    const Box bk = box(k, d->dtype, d->k_stride, d->B, d->H_k, d->N, d->d), bko = box(k_out, d->dtype, d->k_out_stride, d->B, d->H_k, d->N, d->d);
    if ((s = check_no_overlap(bqo, bk, "q_out", "k")) || (s = check_no_overlap(bqo, bko, "q_out", "k_out")) ||
        (s = check_no_overlap(bko, bk, "k_out", "k")) || (s = check_no_overlap(bko, bq, "k_out", "q")))
      return s;
  }
  rn::RotaryCall c;
  c.B = d->B; c.N = d->N; c.Hq = d->H_q; c.Hk = d->H_k; c.d = d->d; c.rot = d->rot; c.dt = d->dtype;
  c.half = d->flags & RN_ROTARY_HALF;
  c.inverse = d->flags & RN_ROTARY_INVERSE;
  c.pos_token = d->flags & RN_ROTARY_POS_TOKEN;
  c.magnitude = d->magnitude; c.pos0 = d->pos0; c.pos = pos; c.theta = d->theta;
  c.qs = d->q_stride; c.ks = d->k_stride; c.qos = d->q_out_stride; c.kos = d->k_out_stride;
  c.q = q; c.k = k; c.q_out = q_out; c.k_out = k_out;
  rn::clear_error();
  return hip_status(rn::launch_rotary(c, static_cast<hipStream_t>(stream)), "rotary launch");
}

rn_status rn_rotary_frequencies(int32_t rot, double base, int32_t kind, double factor, double length, double slow,
                                double fast, double* theta, float* magnitude) {
  if (rot < 2 || rot % 2) return fail(RN_ERR_INVALID_ARG, "rot=%d must be even and >= 2", rot);
  if (rot > rn::kMaxRot) return fail(RN_ERR_UNSUPPORTED, "rot=%d > %d", rot, rn::kMaxRot);
  if (!(base > 1.0 && std::isfinite(base))) return fail(RN_ERR_INVALID_ARG, "base must be finite and > 1");
  if (kind < RN_ROPE_PLAIN || kind > RN_ROPE_BY_PARTS) return fail(RN_ERR_INVALID_ARG, "unknown kind %d", kind);
  if (kind != RN_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
    return fail(RN_ERR_INVALID_ARG, "factor must be finite and >= 1");
  if (kind == RN_ROPE_BASE && rot < 4) return fail(RN_ERR_INVALID_ARG, "RN_ROPE_BASE needs rot >= 4");
  if (kind == RN_ROPE_BY_PARTS &&
      !(length >= 1.0 && std::isfinite(length) && slow >= 0.0 && fast > slow && std::isfinite(fast)))
    return fail(RN_ERR_INVALID_ARG, "RN_ROPE_BY_PARTS needs length >= 1 and 0 <= slow < fast");
  if (!theta || !magnitude) return fail(RN_ERR_INVALID_ARG, "theta/magnitude pointer is NULL");
  const double b = kind == RN_ROPE_BASE ? base * std::pow(factor, double(rot) / (rot - 2)) : base;
  if (!std::isfinite(b)) return fail(RN_ERR_INVALID_ARG, "base * factor^(rot/(rot-2)) is not finite");
  *magnitude = kind == RN_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  for (int j = 0; j < rot / 2; ++j) {
    const double th = std::pow(b, -2.0 * j / rot);
    double keep = 1.0;   // share of the unstretched angle
    if (kind == RN_ROPE_LINEAR) keep = 0.0;
    if (kind == RN_ROPE_BY_PARTS) {
      const double turns = length * th / (2.0 * M_PI);
      keep = std::fmin(1.0, std::fmax(0.0, (turns - slow) / (fast - slow)));
    }
    theta[j] = kind == RN_ROPE_LINEAR ? th / factor
               : kind == RN_ROPE_BY_PARTS ? th * (keep + (1.0 - keep) / factor) : th;
  }
  rn::clear_error();
  return RN_OK;
}

size_t rn_linear_attention_workspace_bytes(const rn_linear_desc* desc) {
  rn::LinCall c;
  if (check_linear(desc, false, &c) != RN_OK) return 0;
  return (rn::lin_ws_bytes(c) + 255) & ~size_t(255);
}

rn_status rn_linear_attention_chunked(const rn_linear_desc* desc, const int32_t* cu_seqlens, const int32_t* lengths,
                                      const int32_t* slots, const void* q, const void* k, const void* v,
                                      const float* log_decay, const float* state_in, float* state_out, void* out,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  rn::LinCall c;
  rn_status s = check_linear(desc, false, &c);
  if (s != RN_OK) return s;
  if ((s = check_linear_ptrs(desc, slots, q, k, v, log_decay, out, &c)) != RN_OK) return s;
  if (desc->T ? !cu_seqlens : cu_seqlens != nullptr)
    return fail(RN_ERR_INVALID_ARG, "cu_seqlens goes with a packed batch (T > 0) and only with one");
  if (desc->T && lengths) return fail(RN_ERR_INVALID_ARG, "a packed batch takes no lengths");
  if (!aligned(cu_seqlens, 4) || !aligned(lengths, 4))
    return fail(RN_ERR_INVALID_ARG, "cu_seqlens and lengths must be 4-byte aligned");
  if (!aligned(state_in, 16) || !aligned(state_out, 16))
    return fail(RN_ERR_INVALID_ARG, "states must be 16-byte aligned");
  if ((s = check_workspace(workspace, workspace_bytes, rn_linear_attention_workspace_bytes(desc))) != RN_OK) return s;
  if ((s = check_apart(desc, c)) != RN_OK) return s;
  c.cu = cu_seqlens; c.lens = lengths; c.state_in = state_in; c.state_out = state_out; c.ws = workspace;
  rn::clear_error();
  return hip_status(rn::launch_linear_chunked(c, static_cast<hipStream_t>(stream)), "linear attention launch");
}

rn_status rn_linear_attention_step(const rn_linear_desc* desc, const int32_t* slots, const void* q, const void* k,
                                   const void* v, const float* log_decay, float* state, void* out, void* stream) {
  rn::LinCall c;
  rn_status s = check_linear(desc, true, &c);
  if (s != RN_OK) return s;
  if ((s = check_linear_ptrs(desc, slots, q, k, v, log_decay, out, &c)) != RN_OK) return s;
  if (!state) return fail(RN_ERR_INVALID_ARG, "state pointer is NULL");
  if (!aligned(state, 16)) return fail(RN_ERR_INVALID_ARG, "state must be 16-byte aligned");
  if ((s = check_apart(desc, c)) != RN_OK) return s;
  c.state_out = state;
  rn::clear_error();
  return hip_status(rn::launch_linear_step(c, static_cast<hipStream_t>(stream)), "linear attention step launch");
}

}  // extern "C"
