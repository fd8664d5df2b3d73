// C ABI of the short convolution and the selective scan: host-side validation and dispatch, before any
// HIP call.
#include <hip/hip_runtime.h>

#include <cstring>

#include "api_checks.h"
#include "rn_kernels.h"
#include "rn_retention.h"

namespace {

using namespace rn;

constexpr int kMaxChannels = 65536;

rn_status check_pair(const int64_t* s, const char* what) {
  for (int i = 0; i < 2; ++i)
    if (s[i] < 0 || s[i] > kMaxStride)
      return fail(RN_ERR_INVALID_ARG, "%s stride %lld outside [0, 2^40]", what, (long long)s[i]);
  return RN_OK;
}

// Sequences, tokens and packed rows of either descriptor.
rn_status check_batch(int32_t S, int32_t N, int32_t D, int64_t T, bool step) {
  if (S < 1 || N < 1 || D < 1) return fail(RN_ERR_INVALID_ARG, "sizes must be >= 1 (S=%d N=%d D=%d)", S, N, D);
  if (S > 65534) return fail(RN_ERR_UNSUPPORTED, "S=%d > 65534", S);
  if (N > (1 << 30)) return fail(RN_ERR_UNSUPPORTED, "N=%d > 2^30", N);
  if (D > kMaxChannels) return fail(RN_ERR_UNSUPPORTED, "D=%d > %d", D, kMaxChannels);
  if (T < 0 || T > INT32_MAX) return fail(RN_ERR_INVALID_ARG, "T=%lld outside [0, 2^31 - 1]", (long long)T);
  if (step && N != 1) return fail(RN_ERR_INVALID_ARG, "the step needs N == 1 (got %d)", N);
  if (step && T) return fail(RN_ERR_INVALID_ARG, "the step takes no packed batch (T=%lld)", (long long)T);
  if (T && N > T) return fail(RN_ERR_INVALID_ARG, "N=%d > T=%lld", N, (long long)T);
  if (!T && int64_t(S) * N > INT32_MAX) return fail(RN_ERR_UNSUPPORTED, "S*N=%lld > 2^31 - 1", (long long)S * N);
  return RN_OK;
}

rn_status check_lists(int64_t T, const int32_t* cu, const int32_t* lengths, const int32_t* slots, int32_t n_slots) {
  if (T ? !cu : cu != nullptr)
    return fail(RN_ERR_INVALID_ARG, "cu_seqlens goes with a packed batch (T > 0) and only with one");
  if (T && lengths) return fail(RN_ERR_INVALID_ARG, "a packed batch takes no lengths");
  if (!aligned(cu, 4) || !aligned(lengths, 4) || !aligned(slots, 4))
    return fail(RN_ERR_INVALID_ARG, "cu_seqlens, lengths and slots must be 4-byte aligned");
  if (slots && n_slots < 1) return fail(RN_ERR_INVALID_ARG, "n_slots=%d must be >= 1", n_slots);
  return RN_OK;
}

// A tensor [S, N, D] (packed: [1, T, D]), or its B and C.
template <class Desc>
Box token_box(const Desc* d, const void* p, const int64_t* s) {
  return Box{p, size_of(d->dtype), {s[0], 0, s[1]}, {d->T ? 1 : d->S, 1, d->T ? d->T : d->N}, d->D};
}
Box group_box(const rn_scan_desc* d, const void* p, const int64_t* s) {
  return Box{p, size_of(d->dtype), {s[0], s[1], s[2]}, {d->T ? 1 : d->S, d->G, d->T ? d->T : d->N}, d->n};
}
rn_status check_distinct(const Box& b, const char* what) {
  return rn::check_distinct(b.s, b.n[0], b.n[1], b.n[2], b.d, what);
}
// Blocks read their inputs while others write.
rn_status check_apart(const Box& out, const Box& in, const char* what, const char* other) {
  if (in.p && in.p == out.p) return fail(RN_ERR_INVALID_ARG, "%s must not be %s", what, other);
  return check_no_overlap(out, in, what, other);
}

// A sequence's state is read and replaced by the same threads: the one buffer in both places is fine, one
// shifted against the other is not.
template <class Desc>
rn_status check_states(const Desc* d, bool slots, rn_dtype dt, int64_t row, const void* out, const void* in, const char* what,
                       const char* other) {
  if (!out || !in) return RN_OK;
  const int64_t n = slots ? d->n_slots : d->S;
  const Box a{out, size_of(dt), {row, 0, 0}, {n, 1, 1}, row}, b{in, size_of(dt), {row, 0, 0}, {n, 1, 1}, row};
  return check_no_overlap(a, b, what, other);
}

// ---- short convolution ----------------------------------------------------------------------

rn_status check_conv(const rn_conv_desc* d, bool step, bool back, rn::ConvCall* c) {
  if (!d) return fail(RN_ERR_INVALID_ARG, "desc is NULL");
  rn_status s = check_batch(d->S, d->N, d->D, d->T, step);
  if (s != RN_OK) return s;
  if (d->K < 1) return fail(RN_ERR_INVALID_ARG, "K=%d must be >= 1", d->K);
  if (d->K > 8) return fail(RN_ERR_UNSUPPORTED, "K=%d > 8", d->K);
  if (!dtype_ok(d->dtype)) return fail(RN_ERR_INVALID_ARG, "unknown dtype (%d)", d->dtype);
  if (d->flags & ~(RN_SEQ_ZERO_REST | RN_CONV_SILU)) return fail(RN_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags);
  if ((s = check_pair(d->x_stride, "x")) || (s = check_pair(d->out_stride, "out")) || (back && (s = check_pair(d->dx_stride, "dx"))) ||
      (s = back ? check_distinct(token_box(d, nullptr, d->dx_stride), "dx") : check_distinct(token_box(d, nullptr, d->out_stride), "out")))
    return s;
  std::memset(c, 0, sizeof(*c));
  c->S = d->S; c->N = d->N; c->D = d->D; c->K = d->K; c->n_slots = d->n_slots; c->T = d->T; c->dt = d->dtype;
  c->silu = d->flags & RN_CONV_SILU; c->zero_rest = d->flags & RN_SEQ_ZERO_REST; c->backward = back; c->step = step;
  c->xs = d->x_stride; c->os = d->out_stride; c->ds = d->dx_stride;
  return RN_OK;
}

rn_status check_conv_ptrs(const rn_conv_desc* d, const float* weight, const float* bias, const void* x, const void* out,
                          const char* what) {
  if (!x || !weight || !out) return fail(RN_ERR_INVALID_ARG, "x/weight/%s pointer is NULL", what);
  rn_status s;
  if ((s = check_elements(x, d->dtype, "x")) || (s = check_elements(out, d->dtype, what)) ||
      (s = check_elements(weight, RN_F32, "weight")) || (s = check_elements(bias, RN_F32, "bias")))
    return s;
  return RN_OK;
}

// 16-byte accesses: whole pieces of channels in every row of every tensor.
bool conv_vectors(const rn::ConvCall& c) {
  const int v = c.dt == RN_BF16 ? 8 : 4;
  auto ok = [&](const void* p, const int64_t* s) { return !p || (aligned(p, 16) && s[0] % v == 0 && s[1] % v == 0); };
  return c.D % v == 0 && ok(c.x, c.xs) && ok(c.out, c.os) && ok(c.dout, c.os) && ok(c.dx, c.ds) && aligned(c.state_in, 16) &&
         aligned(c.state_out, 16) && aligned(c.dstate_out, 16) && aligned(c.dstate_in, 16);
}

// ---- selective scan -------------------------------------------------------------------------

rn_status check_scan(const rn_scan_desc* d, bool step, rn::ScanCall* c) {
  if (!d) return fail(RN_ERR_INVALID_ARG, "desc is NULL");
  rn_status s = check_batch(d->S, d->N, d->D, d->T, step);
  if (s != RN_OK) return s;
  if (d->n < 1 || d->G < 1) return fail(RN_ERR_INVALID_ARG, "sizes must be >= 1 (n=%d G=%d)", d->n, d->G);
  if (d->n > 64) return fail(RN_ERR_UNSUPPORTED, "n=%d > 64", d->n);
  if (d->D % d->G) return fail(RN_ERR_INVALID_ARG, "G=%d must divide D=%d", d->G, d->D);
  if (!dtype_ok(d->dtype)) return fail(RN_ERR_INVALID_ARG, "unknown dtype (%d)", d->dtype);
  if (d->flags & ~(RN_SEQ_ZERO_REST | RN_SCAN_SOFTPLUS)) return fail(RN_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags);
  if ((s = check_pair(d->x_stride, "x")) || (s = check_pair(d->dt_stride, "dt")) || (s = check_pair(d->z_stride, "z")) ||
      (s = check_pair(d->out_stride, "out")) || (s = check_strides(d->b_stride, "B")) || (s = check_strides(d->c_stride, "C")))
    return s;
  std::memset(c, 0, sizeof(*c));
  c->S = d->S; c->N = d->N; c->D = d->D; c->n = d->n; c->G = d->G; c->n_slots = d->n_slots; c->T = d->T; c->type = d->dtype;
  c->softplus = d->flags & RN_SCAN_SOFTPLUS; c->zero_rest = d->flags & RN_SEQ_ZERO_REST;
  c->xs = d->x_stride; c->dts = d->dt_stride; c->zs = d->z_stride; c->os = d->out_stride; c->bs = d->b_stride; c->cs = d->c_stride;
  return RN_OK;
}

rn_status check_scan_ptrs(const rn_scan_desc* d, const void* x, const void* dt, const float* A, const void* B, const void* C,
                          const float* skip, const float* bias, const void* z, rn::ScanCall* c) {
  if (!x || !dt || !A || !B || !C) return fail(RN_ERR_INVALID_ARG, "x/dt/A/B/C pointer is NULL");
  rn_status s;
  if ((s = check_elements(x, d->dtype, "x")) || (s = check_elements(dt, d->dtype, "dt")) || (s = check_elements(A, RN_F32, "A")) ||
      (s = check_elements(B, d->dtype, "B")) || (s = check_elements(C, d->dtype, "C")) || (s = check_elements(skip, RN_F32, "skip")) ||
      (s = check_elements(bias, RN_F32, "bias")) || (s = check_elements(z, d->dtype, "z")))
    return s;
  c->x = x; c->dt = dt; c->A = A; c->b = B; c->c = C; c->skip = skip; c->bias = bias; c->z = z;
  return RN_OK;
}

// States are moved by fours where a channel has whole fours of them, and one by one elsewhere: such states may be any
// slice of a pool.
rn_status check_state_address(const rn_scan_desc* d, const void* p, const char* what) {
  const int n = d->n % 4 == 0 ? 16 : 4;
  if (!aligned(p, n)) return fail(RN_ERR_INVALID_ARG, "%s must be %d-byte aligned", what, n);
  return RN_OK;
}

// `out` (a token gradient) against every input that has rows of tokens.
rn_status check_scan_apart(const rn_scan_desc* d, const rn::ScanCall& c, const Box& out, const char* what) {
  rn_status s;
  if ((s = check_apart(out, token_box(d, c.x, d->x_stride), what, "x")) ||
      (s = check_apart(out, token_box(d, c.dt, d->dt_stride), what, "dt")) ||
      (s = check_apart(out, token_box(d, c.z, d->z_stride), what, "z")) ||
      (s = check_apart(out, group_box(d, c.b, d->b_stride), what, "B")) ||
      (s = check_apart(out, group_box(d, c.c, d->c_stride), what, "C")))
    return s;
  return RN_OK;
}

rn_status check_scan_out(const rn_scan_desc* d, const rn::ScanCall& c, const void* out) {
  if (!out) return fail(RN_ERR_INVALID_ARG, "out pointer is NULL");
  const Box b = token_box(d, out, d->out_stride);
  rn_status s;
  if ((s = check_elements(out, d->dtype, "out")) || (s = check_distinct(b, "out"))) return s;
  return check_scan_apart(d, c, b, "out");
}

}  // namespace

extern "C" {

rn_status rn_short_conv(const rn_conv_desc* desc, const int32_t* cu_seqlens, const int32_t* lengths, const int32_t* slots,
                        const void* x, const float* weight, const float* bias, const void* state_in, void* state_out,
                        void* out, void* stream) {
  rn::ConvCall c;
  rn_status s = check_conv(desc, false, false, &c);
  if (s != RN_OK) return s;
  if ((s = check_conv_ptrs(desc, weight, bias, x, out, "out")) || (s = check_lists(desc->T, cu_seqlens, lengths, slots, desc->n_slots)) ||
      (s = check_elements(state_in, desc->dtype, "state_in")) || (s = check_elements(state_out, desc->dtype, "state_out")) ||
      (s = check_states(desc, slots, desc->dtype, int64_t(desc->K - 1) * desc->D, state_out, state_in, "state_out", "state_in")) ||
      (s = check_apart(token_box(desc, out, desc->out_stride), token_box(desc, x, desc->x_stride), "out", "x")))
    return s;
  c.cu = cu_seqlens; c.lens = lengths; c.slots = slots; c.x = x; c.w = weight; c.b = bias; c.out = out;
  c.state_in = state_in; c.state_out = state_out;
  c.vec = conv_vectors(c);
  rn::clear_error();
  return hip_status(rn::launch_short_conv(c, static_cast<hipStream_t>(stream)), "short convolution launch");
}

rn_status rn_short_conv_step(const rn_conv_desc* desc, const int32_t* slots, const void* x, const float* weight,
                             const float* bias, void* state, void* out, void* stream) {
  rn::ConvCall c;
  rn_status s = check_conv(desc, true, false, &c);
  if (s != RN_OK) return s;
  if ((s = check_conv_ptrs(desc, weight, bias, x, out, "out")) || (s = check_lists(0, nullptr, nullptr, slots, desc->n_slots)) ||
      (s = check_elements(state, desc->dtype, "state")) ||
      (s = check_apart(token_box(desc, out, desc->out_stride), token_box(desc, x, desc->x_stride), "out", "x")))
    return s;
  if (!state && desc->K > 1) return fail(RN_ERR_INVALID_ARG, "state pointer is NULL");
  c.slots = slots; c.x = x; c.w = weight; c.b = bias; c.out = out; c.state_in = state; c.state_out = state;
  c.vec = conv_vectors(c);
  rn::clear_error();
  return hip_status(rn::launch_short_conv(c, static_cast<hipStream_t>(stream)), "short convolution step launch");
}

size_t rn_short_conv_backward_workspace_bytes(const rn_conv_desc* desc) {
  rn::ConvCall c;
  if (check_conv(desc, false, true, &c) != RN_OK) return 0;
  return (rn::conv_backward_ws_bytes(c) + 255) & ~size_t(255);
}

rn_status rn_short_conv_backward(const rn_conv_desc* desc, const int32_t* cu_seqlens, const int32_t* lengths, const void* dout,
                                 const void* x, const float* weight, const float* bias, const void* state_in,
                                 const float* dstate_out, void* dx, float* dweight, float* dbias, float* dstate_in,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  rn::ConvCall c;
  rn_status s = check_conv(desc, false, true, &c);
  if (s != RN_OK) return s;
  if (!dout) return fail(RN_ERR_INVALID_ARG, "dout pointer is NULL");
  const Box bd = token_box(desc, dx, desc->dx_stride);
  if ((s = check_conv_ptrs(desc, weight, bias, x, dx, "dx")) || (s = check_lists(desc->T, cu_seqlens, lengths, nullptr, 0)) ||
      (s = check_elements(dout, desc->dtype, "dout")) || (s = check_elements(state_in, desc->dtype, "state_in")) ||
      (s = check_elements(dstate_out, RN_F32, "dstate_out")) || (s = check_elements(dstate_in, RN_F32, "dstate_in")) ||
      (s = check_elements(dweight, RN_F32, "dweight")) || (s = check_elements(dbias, RN_F32, "dbias")) ||
      (s = check_apart(bd, token_box(desc, x, desc->x_stride), "dx", "x")) ||
      (s = check_apart(bd, token_box(desc, dout, desc->out_stride), "dx", "dout")))
    return s;
  if (dstate_in && dstate_in == dstate_out) return fail(RN_ERR_INVALID_ARG, "dstate_in must not be dstate_out");
  if ((s = check_states(desc, false, RN_F32, int64_t(desc->K - 1) * desc->D, dstate_in, dstate_out, "dstate_in", "dstate_out"))) return s;
  if ((dweight || dbias) && (s = check_workspace(workspace, workspace_bytes, rn_short_conv_backward_workspace_bytes(desc)))) return s;
  c.cu = cu_seqlens; c.lens = lengths; c.x = x; c.w = weight; c.b = bias; c.state_in = state_in; c.dout = dout; c.dx = dx;
  c.dstate_out = dstate_out; c.dstate_in = dstate_in; c.dw = dweight; c.db = dbias; c.ws = workspace;
  c.vec = conv_vectors(c);
  rn::clear_error();
  return hip_status(rn::launch_short_conv(c, static_cast<hipStream_t>(stream)), "short convolution backward launch");
}

size_t rn_selective_scan_workspace_bytes(const rn_scan_desc* desc) {
  rn::ScanCall c;
  if (check_scan(desc, false, &c) != RN_OK) return 0;
  return (rn::scan_ws_bytes(c) + 255) & ~size_t(255);
}

rn_status rn_selective_scan_chunked(const rn_scan_desc* desc, const int32_t* cu_seqlens, const int32_t* lengths,
                                    const int32_t* slots, const void* x, const void* dt, const float* A, const void* B,
                                    const void* C, const float* skip, const float* bias, const void* z, const float* state_in,
                                    float* state_out, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  rn::ScanCall c;
  rn_status s = check_scan(desc, false, &c);
  if (s != RN_OK) return s;
  if ((s = check_scan_ptrs(desc, x, dt, A, B, C, skip, bias, z, &c)) || (s = check_scan_out(desc, c, out)) ||
      (s = check_lists(desc->T, cu_seqlens, lengths, slots, desc->n_slots)))
    return s;
  if ((s = check_state_address(desc, state_in, "state_in")) || (s = check_state_address(desc, state_out, "state_out"))) return s;
  if ((s = check_states(desc, slots, RN_F32, int64_t(desc->D) * desc->n, state_out, state_in, "state_out", "state_in"))) return s;
  if ((s = check_workspace(workspace, workspace_bytes, rn_selective_scan_workspace_bytes(desc)))) return s;
  c.cu = cu_seqlens; c.lens = lengths; c.slots = slots; c.state_in = state_in; c.state_out = state_out; c.out = out; c.ws = workspace;
  rn::clear_error();
  return hip_status(rn::launch_selective_scan(c, static_cast<hipStream_t>(stream)), "selective scan launch");
}

rn_status rn_selective_scan_step(const rn_scan_desc* desc, const int32_t* slots, const void* x, const void* dt, const float* A,
                                 const void* B, const void* C, const float* skip, const float* bias, const void* z, float* state,
                                 void* out, void* stream) {
  rn::ScanCall c;
  rn_status s = check_scan(desc, true, &c);
  if (s != RN_OK) return s;
  if ((s = check_scan_ptrs(desc, x, dt, A, B, C, skip, bias, z, &c)) || (s = check_scan_out(desc, c, out)) ||
      (s = check_lists(0, nullptr, nullptr, slots, desc->n_slots)))
    return s;
  if (!state) return fail(RN_ERR_INVALID_ARG, "state pointer is NULL");
  if ((s = check_state_address(desc, state, "state"))) return s;
  c.slots = slots; c.state_in = state; c.state_out = state; c.out = out;
  rn::clear_error();
  return hip_status(rn::launch_selective_step(c, static_cast<hipStream_t>(stream)), "selective scan step launch");
}

size_t rn_selective_scan_backward_workspace_bytes(const rn_scan_desc* desc) {
  rn::ScanCall c;
  if (check_scan(desc, false, &c) != RN_OK) return 0;
  return (rn::scan_backward_ws_bytes(c) + 255) & ~size_t(255);
}

rn_status rn_selective_scan_backward(const rn_scan_desc* desc, const rn_scan_grad_desc* grads, const int32_t* cu_seqlens,
                                     const int32_t* lengths, const void* dout, const void* x, const void* dt, const float* A,
                                     const void* B, const void* C, const float* skip, const float* bias, const void* z,
                                     const float* state_in, const float* dstate_out, void* dx, void* ddt, float* dA, void* dB,
                                     void* dC, float* dskip, float* dbias, void* dz, float* dstate_in, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  rn::ScanCall c;
  rn_status s = check_scan(desc, false, &c);
  if (s != RN_OK) return s;
  if (!grads) return fail(RN_ERR_INVALID_ARG, "grads is NULL");
  if ((s = check_scan_ptrs(desc, x, dt, A, B, C, skip, bias, z, &c)) || (s = check_lists(desc->T, cu_seqlens, lengths, nullptr, 0)))
    return s;
  if (!dout || !dx || !ddt || !dA || !dB || !dC) return fail(RN_ERR_INVALID_ARG, "dout/dx/ddt/dA/dB/dC pointer is NULL");
  if ((z != nullptr) != (dz != nullptr)) return fail(RN_ERR_INVALID_ARG, "dz goes with z");
  const Box in = token_box(desc, dout, desc->out_stride);
  struct { Box b; const int64_t* strides; const char* name; bool heads; } outs[5] = {
      {token_box(desc, dx, grads->dx_stride), grads->dx_stride, "dx", false},
      {token_box(desc, ddt, grads->ddt_stride), grads->ddt_stride, "ddt", false},
      {group_box(desc, dB, grads->db_stride), grads->db_stride, "dB", true},
      {group_box(desc, dC, grads->dc_stride), grads->dc_stride, "dC", true},
      {token_box(desc, dz, grads->dz_stride), grads->dz_stride, "dz", false}};
  if ((s = check_elements(dout, desc->dtype, "dout"))) return s;
  for (int i = 0; i < (dz ? 5 : 4); ++i) {
    const auto& o = outs[i];
    if ((s = o.heads ? check_strides(o.strides, o.name) : check_pair(o.strides, o.name)) || (s = check_elements(o.b.p, desc->dtype, o.name)) ||
        (s = check_distinct(o.b, o.name)) || (s = check_scan_apart(desc, c, o.b, o.name)) || (s = check_apart(o.b, in, o.name, "dout")))
      return s;
    for (int j = 0; j < i; ++j)
      if ((s = check_apart(o.b, outs[j].b, o.name, outs[j].name))) return s;
  }
  for (const float* p : {static_cast<const float*>(dA), static_cast<const float*>(dskip), static_cast<const float*>(dbias)})
    if ((s = check_elements(p, RN_F32, "dA/dskip/dbias"))) return s;
  for (const float* p : {state_in, dstate_out, static_cast<const float*>(dstate_in)})
    if ((s = check_state_address(desc, p, "a state or its gradient"))) return s;
  if (dstate_in && (dstate_in == dstate_out || dstate_in == state_in))
    return fail(RN_ERR_INVALID_ARG, "dstate_in must be no other operand");
  for (const float* p : {state_in, dstate_out})
    if ((s = check_states(desc, false, RN_F32, int64_t(desc->D) * desc->n, dstate_in, p, "dstate_in", "a state"))) return s;
  if ((s = check_workspace(workspace, workspace_bytes, rn_selective_scan_backward_workspace_bytes(desc)))) return s;
  c.cu = cu_seqlens; c.lens = lengths; c.state_in = state_in; c.ws = workspace;
  rn::ScanGrads g;
  g.dxs = grads->dx_stride; g.ddts = grads->ddt_stride; g.dzs = grads->dz_stride; g.dbs = grads->db_stride; g.dcs = grads->dc_stride;
  g.dout = dout; g.dstate_out = dstate_out; g.dx = dx; g.ddt = ddt; g.dz = dz; g.db = dB; g.dc = dC;
  g.dA = dA; g.dskip = dskip; g.dbias = dbias; g.dstate_in = dstate_in;
  rn::clear_error();
  return hip_status(rn::launch_selective_backward(c, g, static_cast<hipStream_t>(stream)), "selective scan backward launch");
}

}  // extern "C"
