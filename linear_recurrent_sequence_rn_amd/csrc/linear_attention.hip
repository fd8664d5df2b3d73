// Linear attention with a decay per head and token, in float32:
//     S_t = exp(g_t) S_{t-1} + k_t^T v_t,     o_t = scale q_t S_t.
//
// lin_step: one token a sequence. Bound by HBM: the float32 state is read and written once.
// lin_recurrent: prompts of any type and head size by the recurrence itself, token by token,
// the state in registers. Bound by the vector units (three operations a state element and token)
// and by the chain of tokens where few states leave a compute unit one block (padded float32
// batch of 3 sequences of up to 2001 tokens, 5 heads of 48 x 81: 39 us, of which the scan is 8).
// Long sequences are cut into segments: one pass gives the state each segment adds on its own,
// lin_scan carries the states over the segments, a second pass gives the outputs; the same three
// passes carry the matrix-core kernel's segments.
#include <algorithm>

#include "linear_attention.h"

namespace rn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---- one token a sequence ---------------------------------------------------------------
// A block of NT threads owns NQ * VEC columns of one (sequence, head) state; thread (group,
// column vector) takes rows group, group + G, ... in batches of 8, the next batch's loads issued
// before the present one is updated. Non-temporal: a batch's states are larger than the caches
// and are read once a step. FULL: every thread has a column and every batch its rows, so that
// no load hangs on a condition (128 states of 16 heads of 256 x 512: 357 us, 6.0 TB/s; with
// conditions and half the columns a block 460 us).
constexpr int kBatch = 8;

template <int IN, int OUT, int VEC, int NQ, int NT, bool FULL>
__global__ void __launch_bounds__(NT) lin_step(LinArgs a, int slices) {
  constexpr int G = NT / NQ;
  constexpr int W = NQ * VEC;
  __shared__ float qh[kMaxDk];
  __shared__ float kh[kMaxDk];
  __shared__ float part[G * W];
  const int h = blockIdx.x / slices, c0 = (blockIdx.x - h * slices) * W;
  const int s = blockIdx.y, tid = threadIdx.x;
  const int cq = tid % NQ, grp = tid / NQ;
  const int slot = lin_slot(a, s);
  const int64_t oo = s * a.os[0] + h * a.os[1] + c0;
  const int nc = min(W, a.dv - c0);
  if (slot < 0) {
    for (int c = tid; c < nc; c += NT) Elem<OUT>::store(a.out, oo + c, 0.f);
    return;
  }
  const int64_t qo = s * a.qs[0] + h / (a.H / a.Hq) * a.qs[1];
  const int64_t ko = s * a.ks[0] + h / (a.H / a.Hk) * a.ks[1];
  const int64_t vo = s * a.vs[0] + h / (a.H / a.Hv) * a.vs[1] + c0;
  const int dk = a.dk, dv = a.dv;
  const bool col = FULL || cq * VEC < nc;
  float* S = a.state_out + (static_cast<int64_t>(slot) * a.H + h) * dk * dv + c0 + cq * VEC;
  auto load = [&](int d0, float (*x)[VEC]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int d = d0 + u * G;
      if (FULL || (col && d < dk)) {
        if constexpr (VEC == 4) {
          const f32x4 y = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(S + static_cast<int64_t>(d) * dv));
          x[u][0] = y.x; x[u][1] = y.y; x[u][2] = y.z; x[u][3] = y.w;
        } else {
          x[u][0] = __builtin_nontemporal_load(S + static_cast<int64_t>(d) * dv);
        }
      }
    }
  };
  float xa[kBatch][VEC], xb[kBatch][VEC];
  load(grp, xa);
  for (int d = tid; d < dk; d += NT) {
    qh[d] = Elem<IN>::load(a.q, qo + d);
    kh[d] = Elem<IN>::load(a.k, ko + d);
  }
  const float dec = expf(a.g[s * a.gs[0] + h * a.gs[1]]);
  float vr[VEC], acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    vr[i] = col ? Elem<IN>::load(a.v, vo + cq * VEC + i) : 0.f;
    acc[i] = 0.f;
  }
  auto update = [&](int d0, float (*x)[VEC]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int d = d0 + u * G;
      if (FULL || (col && d < dk)) {
        const float kd = kh[d], qd = qh[d];
        float y[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          y[i] = fmaf(dec, x[u][i], kd * vr[i]);
          acc[i] = fmaf(qd, y[i], acc[i]);
        }
        if constexpr (VEC == 4) {
          const f32x4 z = {y[0], y[1], y[2], y[3]};
          __builtin_nontemporal_store(z, reinterpret_cast<f32x4*>(S + static_cast<int64_t>(d) * dv));
        } else {
          __builtin_nontemporal_store(y[0], S + static_cast<int64_t>(d) * dv);
        }
      }
    }
  };
  __syncthreads();
  for (int d0 = grp; d0 < dk; d0 += 2 * G * kBatch) {
    // (with FULL, d_k - d0 is a multiple of a batch plus the group: these tests are uniform)
    const bool second = d0 - grp + G * kBatch < dk, third = d0 - grp + 2 * G * kBatch < dk;
    if (second) load(d0 + G * kBatch, xb);
    update(d0, xa);
    if (third) load(d0 + 2 * G * kBatch, xa);
    if (second) update(d0 + G * kBatch, xb);
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) part[grp * W + cq * VEC + i] = acc[i];
  __syncthreads();
  if constexpr (G > 8 && W < NT) {          // many groups: all threads add a few, then the columns' own
    constexpr int T = NT / W, P = G / T;
    const int c = tid % W, i0 = tid / W * P;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) o += part[(i0 + i) * W + c];
    __syncthreads();
    part[tid / W * W + c] = o;
    __syncthreads();
    if (tid < nc) {
      o = 0.f;
#pragma unroll
      for (int i = 0; i < T; ++i) o += part[i * W + tid];
      Elem<OUT>::store(a.out, oo + tid, a.scale * o);
    }
  } else {
    for (int c = tid; c < nc; c += NT) {
      float o = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) o += part[i * W + c];
      Elem<OUT>::store(a.out, oo + c, a.scale * o);
    }
  }
}

// ---- prompts by the recurrence ------------------------------------------------------------
// A block owns 64 columns of one head's state over one segment of one sequence, in registers: wave
// w holds the rows [w RW, (w+1) RW), and each of its lanes RW / 4 rows of 4 neighbouring columns
// (lane = 4 column quad + row group), so that 16 bytes from LDS feed 16 state elements (rows past
// d_k stay zero). Tokens come in blocks of 16 through LDS, the next block's loads in flight
// meanwhile; the four row groups' shares of an output meet by DPP, the waves' in LDS. (One column
// and RW rows a lane read 16 bytes of LDS for 4 elements and were bound by that: 12 x 16 heads of
// 212 bf16 tokens, 128 x 81: 218 -> 94 us; 3 heads of 1169 float32 tokens, 192 x 81: 135 -> 65.)
constexpr int kTok = 16;
constexpr int kCols = 64;

// the value of the lane whose number differs in bit B of a quad
template <int B>
__device__ __forceinline__ float quad_swap(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), B == 1 ? 0xB1 : 0x4E, 0xf, 0xf, true));
}

template <int IN, int OUT, int RW, LinMode MODE>
__global__ void __launch_bounds__(256) lin_recurrent(LinArgs a) {
  constexpr int D = 4 * RW;
  constexpr int E = kTok * D / 256;       // q (or k) elements a thread stages
  __shared__ float qt[kTok][D];
  __shared__ float kt[kTok][D];
  __shared__ float vt[kTok][kCols];
  __shared__ float gt[kTok];
  __shared__ float part[4][kTok][kCols];
  int h, c0;
  lin_block(a, blockIdx.x, &h, &c0);
  c0 *= kCols;
  int seg, s;
  if (!lin_place(a, &s, &seg)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nc = min(kCols, a.dv - c0);
  int64_t row0, own;
  int len;
  lin_span(a, s, &row0, &len, &own);
  if (MODE != kLinState && a.zero_rest) lin_zero_rest<OUT>(a, s, seg, h, c0, nc, row0, len, own);
  if (s == a.S) return;
  const int t0 = min(seg, a.n_seg) * a.seg_len;
  const int t1 = min(len, t0 + a.seg_len);
  const int slot = lin_slot(a, s);
  const int64_t sh = static_cast<int64_t>(a.dk) * a.dv;
  const bool keep = a.state_out && slot >= 0;
  const bool one = len <= a.seg_len;      // (always, where kLinWhole is the only pass)
  if (t0 >= t1 && !(MODE == kLinWhole && seg == 0 && keep)) return;
  if (MODE == kLinState && t1 == len && (!keep || (a.flat && one))) return;   // nobody reads the last segment's state

  constexpr int RL = RW / 4;
  const int sub = lane & 3, cq = lane & ~3;
  auto row = [&](int r) { return wave * RW + (r >> 2) * 16 + sub * 4 + (r & 3); };
  const bool quads = a.dv % 4 == 0;   // (states are 16-byte aligned)
  float S[RL][4];
  {
    const float* from = MODE == kLinState ? nullptr
                        : MODE == kLinOut || !one ? a.seg_state + (lin_segment(a, s, row0, seg) * a.H + h) * sh
                        : a.state_in && slot >= 0 ? a.state_in + (static_cast<int64_t>(slot) * a.H + h) * sh : nullptr;
#pragma unroll
    for (int r = 0; r < RL; ++r) {
      const int d = row(r);
      f32x4 x = {};
      if (from && d < a.dk) {
        const float* p = from + (static_cast<int64_t>(d) * a.dv + c0 + cq);
        if (quads) {
          if (cq < nc) x = *reinterpret_cast<const f32x4*>(p);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (cq + c < nc) x[c] = p[c];
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) S[r][c] = x[c];
    }
  }
  const int64_t qo = lin_base(a, a.qs, s, row0) + h / (a.H / a.Hq) * a.qs[1];
  const int64_t ko = lin_base(a, a.ks, s, row0) + h / (a.H / a.Hk) * a.ks[1];
  const int64_t vo = lin_base(a, a.vs, s, row0) + h / (a.H / a.Hv) * a.vs[1] + c0;
  const int64_t go = lin_base(a, a.gs, s, row0) + h * a.gs[1];
  const int64_t oo = lin_base(a, a.os, s, row0) + h * a.os[1] + c0;

  float rq[E], rk[E], rv[kTok * kCols / 256], rg = 0.f;
  // every load is of a token and an element that exist; what should be zero is made so after it
  auto fetch = [&](int t) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = tid + 256 * e, tt = min(t + i / D, t1 - 1), d = min(i % D, a.dk - 1);
      if constexpr (MODE != kLinState) rq[e] = Elem<IN>::load(a.q, qo + tt * a.qs[2] + d);
      rk[e] = Elem<IN>::load(a.k, ko + tt * a.ks[2] + d);
    }
#pragma unroll
    for (int e = 0; e < kTok * kCols / 256; ++e) {
      const int i = tid + 256 * e, tt = min(t + i / kCols, t1 - 1), c = min(i % kCols, nc - 1);
      rv[e] = Elem<IN>::load(a.v, vo + tt * a.vs[2] + c);
    }
    rg = a.g[go + min(t + (tid & (kTok - 1)), t1 - 1) * a.gs[2]];
  };
  double gsum = 0.0;
  if (t0 < t1) fetch(t0);
  for (int t = t0; t < t1; t += kTok) {
    const int n = min(kTok, t1 - t);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = tid + 256 * e;
      const bool ok = i / D < n && i % D < a.dk;
      if constexpr (MODE != kLinState) qt[i / D][i % D] = ok ? rq[e] : 0.f;
      kt[i / D][i % D] = ok ? rk[e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < kTok * kCols / 256; ++e) {
      const int i = tid + 256 * e;
      vt[i / kCols][i % kCols] = i / kCols < n && i % kCols < nc ? rv[e] : 0.f;
    }
    if (tid < kTok) {
      gt[tid] = tid < n ? expf(rg) : 1.f;
      gsum += tid < n ? rg : 0.f;
    }
    __syncthreads();
    if (t + kTok < t1) fetch(t + kTok);
    // A token's values are read from LDS while the one before it is worked on. (Tokens behind the
    // last have decay 1 and k = q = v = 0, and change nothing.)
    struct Token { float4 k[RL / 4], q[RL / 4], v; float dec; } ta, tb;
    auto read = [&](int i, Token& x) {
      x.dec = gt[i];
      x.v = *reinterpret_cast<const float4*>(&vt[i][cq]);
#pragma unroll
      for (int j = 0; j < RL / 4; ++j) {
        x.k[j] = *reinterpret_cast<const float4*>(&kt[i][wave * RW + 16 * j + 4 * sub]);
        if constexpr (MODE != kLinState) x.q[j] = *reinterpret_cast<const float4*>(&qt[i][wave * RW + 16 * j + 4 * sub]);
      }
    };
    auto work = [&](int i, const Token& x) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const float v[4] = {x.v.x, x.v.y, x.v.z, x.v.w};
#pragma unroll
      for (int j = 0; j < RL / 4; ++j) {
        const float k[4] = {x.k[j].x, x.k[j].y, x.k[j].z, x.k[j].w};
        const float q[4] = {x.q[j].x, x.q[j].y, x.q[j].z, x.q[j].w};
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float& st = S[4 * j + r][c];
            st = fmaf(x.dec, st, k[r] * v[c]);
            if constexpr (MODE != kLinState) acc[c] = fmaf(q[r], st, acc[c]);
          }
      }
      if constexpr (MODE != kLinState) {
        // the sum over the quad's lanes; lane i of a quad keeps column i
        const bool b1 = lane & 2, b0 = lane & 1;
        const float u0 = (b1 ? acc[2] : acc[0]) + quad_swap<2>(b1 ? acc[0] : acc[2]);
        const float u1 = (b1 ? acc[3] : acc[1]) + quad_swap<2>(b1 ? acc[1] : acc[3]);
        part[wave][i][lane] = (b0 ? u1 : u0) + quad_swap<1>(b0 ? u0 : u1);
      }
    };
    read(0, ta);
#pragma unroll 2
    for (int i = 0; i < kTok; i += 2) {
      read(i + 1, tb);
      __builtin_amdgcn_sched_barrier(0);
      work(i, ta);
      read(i + 2 < kTok ? i + 2 : 0, ta);
      __builtin_amdgcn_sched_barrier(0);
      work(i + 1, tb);
    }
    __syncthreads();
    if constexpr (MODE != kLinState) {
#pragma unroll
      for (int e = 0; e < kTok / 4; ++e) {
        const int i = wave + 4 * e;
        if (i < n && lane < nc)
          Elem<OUT>::store(a.out, oo + (t + i) * a.os[2] + lane,
                           a.scale * ((part[0][i][lane] + part[1][i][lane]) + (part[2][i][lane] + part[3][i][lane])));
      }
    }
  }
  float* to = nullptr;
  if (MODE == kLinWhole && keep && one) to = a.state_out + (static_cast<int64_t>(slot) * a.H + h) * sh;
  if (MODE == kLinState) {
    const int64_t i = lin_segment(a, s, row0, seg) * a.H + h;
    to = a.seg_state + i * sh;
    // (thread t holds the sum of tokens t, t + 16, ... of the segment)
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) gsum += __shfl_xor(gsum, o, 16);
    if (c0 == 0 && tid == 0) a.seg_decay[i] = expf(static_cast<float>(gsum));
  }
  if (to) {
#pragma unroll
    for (int r = 0; r < RL; ++r) {
      const int d = row(r);
      if (d < a.dk) {
        float* p = to + (static_cast<int64_t>(d) * a.dv + c0 + cq);
        if (quads) {
          const f32x4 x = {S[r][0], S[r][1], S[r][2], S[r][3]};
          if (cq < nc) *reinterpret_cast<f32x4*>(p) = x;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (cq + c < nc) p[c] = S[r][c];
        }
      }
    }
  }
}

// ---- states over the segments ---------------------------------------------------------------
// V neighbouring state elements a thread: the segments' own states become the states they start
// from, and the last one the final state.
template <int V>
__global__ void __launch_bounds__(256) lin_scan(LinArgs a) {
  typedef float fv __attribute__((ext_vector_type(V)));
  const int h = blockIdx.y;
  // In a flat grid block m - 1 has the sequence of more than one segment that starts in front of
  // token row m L, the first such row behind its start, and ends behind it.
  const int64_t m = blockIdx.z + int64_t(1);
  const int s = a.flat ? lin_last(a, [&](int i) { return lin_first(a, i) <= m * a.seg_len; }) : static_cast<int>(blockIdx.z);
  if (s == a.S) return;
  const int64_t sh = static_cast<int64_t>(a.dk) * a.dv;
  const int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
  if (e >= sh) return;
  int64_t row0, own;
  int len;
  lin_span(a, s, &row0, &len, &own);
  if (a.flat && (len <= a.seg_len || row0 / a.seg_len + 1 != m)) return;
  const int slot = lin_slot(a, s);
  const int n = (len + a.seg_len - 1) / a.seg_len;
  const int64_t at = (static_cast<int64_t>(slot) * a.H + h) * sh + e;
  fv x = {};
  if (a.state_in && slot >= 0) x = *reinterpret_cast<const fv*>(a.state_in + at);
  const int64_t first = lin_segment(a, s, row0, 0) * a.H + h;
  const bool last = a.state_out && slot >= 0;
  float* p = a.seg_state + first * sh + e;
  const float* d = a.seg_decay + first;
  const int64_t ps = sh * a.H;
  // eight segments' states in flight
  for (int g = 0; g < n; g += 8) {
    fv u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g + i < n && (last || g + i + 1 < n)) u[i] = *reinterpret_cast<const fv*>(p + (g + i) * ps);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (g + i < n) {
        *reinterpret_cast<fv*>(p + (g + i) * ps) = x;
        if (last || g + i + 1 < n) {
          const float dec = d[static_cast<int64_t>(g + i) * a.H];
#pragma unroll
          for (int v = 0; v < V; ++v) x[v] = fmaf(dec, x[v], u[i][v]);
        }
      }
  }
  if (last) *reinterpret_cast<fv*>(a.state_out + at) = x;
}

template <int IN, int OUT, LinMode MODE>
hipError_t launch_recurrent_t(const LinArgs& a, hipStream_t st) {
  const int slices = (a.dv + kCols - 1) / kCols;
  const bool rest = a.T > 0 && a.zero_rest && MODE != kLinState;
  const dim3 grid = lin_grid(a, a.H * slices, rest);
  const int rw = (a.dk + 3) / 4;
  if (rw <= 16) hipLaunchKernelGGL((lin_recurrent<IN, OUT, 16, MODE>), grid, dim3(256), 0, st, a);
  else if (rw <= 32) hipLaunchKernelGGL((lin_recurrent<IN, OUT, 32, MODE>), grid, dim3(256), 0, st, a);
  else if (rw <= 48) hipLaunchKernelGGL((lin_recurrent<IN, OUT, 48, MODE>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lin_recurrent<IN, OUT, 64, MODE>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <LinMode MODE>
hipError_t launch_recurrent(const LinArgs& a, int in_dt, int out_dt, hipStream_t st) {
  if (in_dt == RN_F32)
    return out_dt == RN_F32 ? launch_recurrent_t<RN_F32, RN_F32, MODE>(a, st) : launch_recurrent_t<RN_F32, RN_BF16, MODE>(a, st);
  return out_dt == RN_F32 ? launch_recurrent_t<RN_BF16, RN_F32, MODE>(a, st) : launch_recurrent_t<RN_BF16, RN_BF16, MODE>(a, st);
}

template <int IN, int OUT>
hipError_t launch_step_t(const LinArgs& a, hipStream_t st) {
  // Columns a block: as many as the row has (long runs of one state row), but fewer where
  // that leaves the chip's 256 CUs without two blocks each (states are independent by column).
  const int64_t states = static_cast<int64_t>(a.S) * a.H;
#define RN_STEP(VEC, NQ, NT, FULL)                                                                  \
  do {                                                                                              \
    const int slices = (a.dv + VEC * NQ - 1) / (VEC * NQ);                                          \
    hipLaunchKernelGGL((lin_step<IN, OUT, VEC, NQ, NT, FULL>), dim3(a.H * slices, a.S), dim3(NT), 0, st, a, slices); \
    return hipGetLastError();                                                                       \
  } while (0)
  if (a.dv % 4 == 0) {
    if (states >= 512) {
      if (a.dv == 512 && a.dk % 32 == 0) RN_STEP(4, 128, 512, true);
      if (a.dv == 256 && a.dk % 64 == 0) RN_STEP(4, 64, 512, true);
      if (a.dv == 128 && a.dk % 64 == 0) RN_STEP(4, 32, 256, true);
      if (a.dv == 64 && a.dk % 128 == 0) RN_STEP(4, 16, 256, true);
    }
    if (a.dv > 128 && states * ((a.dv + 255) / 256) >= 512) RN_STEP(4, 64, 256, false);
    if (a.dv > 64 && states * ((a.dv + 127) / 128) >= 512) RN_STEP(4, 32, 256, false);
    if (a.dv > 16 && states * ((a.dv + 63) / 64) >= 512) RN_STEP(4, 16, 256, false);
    RN_STEP(4, 4, 256, false);
  }
  RN_STEP(1, 64, 256, false);
#undef RN_STEP
}

LinArgs lin_args(const LinCall& c) {
  LinArgs a;
  a.S = c.S; a.N = c.N; a.H = c.H; a.Hq = c.Hq; a.Hk = c.Hk; a.Hv = c.Hv; a.dk = c.dk; a.dv = c.dv;
  a.n_slots = c.n_slots; a.T = c.T; a.scale = c.scale; a.zero_rest = c.zero_rest;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = c.qs[i]; a.ks[i] = c.ks[i]; a.vs[i] = c.vs[i]; a.gs[i] = c.gs[i]; a.os[i] = c.os[i];
  }
  a.cu = c.cu; a.lens = c.lens; a.slots = c.slots;
  a.q = c.q; a.k = c.k; a.v = c.v; a.g = c.g; a.state_in = c.state_in; a.state_out = c.state_out; a.out = c.out;
  a.seg_len = c.N; a.n_seg = 1; a.flat = false; a.seg_state = nullptr; a.seg_decay = nullptr;
  return a;
}

// Matrix cores: bf16 in and out, head sizes and rows in whole 16-byte pieces. (The pointers are
// not known when the workspace is sized: a call with an unaligned one runs the recurrence on
// the same segments.)
bool mfma_shape(const LinCall& c) {
  bool ok = !c.generic && c.in_dt == RN_BF16 && c.out_dt == RN_BF16 && c.dk % 8 == 0 && c.dv % 8 == 0;
  for (const int64_t* s : {c.qs, c.ks, c.vs, c.os})
    for (int i = 0; i < 3; ++i) ok = ok && s[i] % 8 == 0;
  return ok;
}
bool mfma_call(const LinCall& c) {
  bool ok = mfma_shape(c);
  for (const void* p : {c.q, c.k, c.v, static_cast<const void*>(c.out)}) ok = ok && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  return ok;
}

// Tokens a segment, and how many segments the longest sequence has: one where the sequences and
// heads fill the chip by themselves; else enough that the blocks of all segments do. Cutting
// costs a second pass over the tokens for the states and the scan over them, so a longest
// sequence of less than three segments stays whole.
void segments(const LinCall& c, int* len, int* n) {
  const bool mfma = mfma_shape(c);
  const int64_t per = mfma ? lin_mfma_blocks(lin_args(c)) : static_cast<int64_t>(c.H) * ((c.dv + kCols - 1) / kCols);
  const int64_t tokens = c.T > 0 ? std::min<int64_t>(c.T, static_cast<int64_t>(c.S) * c.N) : static_cast<int64_t>(c.S) * c.N;
  // blocks the 256 CUs hold at once, by their LDS and registers
  const int64_t want = 256 * (!mfma || c.dk <= 64 ? 3 : c.dk <= 128 ? 2 : 1);
  int64_t L = std::max<int64_t>((tokens * per / want + 63) / 64 * 64, mfma ? 256 : 64);
  if (3 * L > c.N) L = c.N;
  L = std::max<int64_t>(L, (c.N + 65534) / 65535);
  L = (L + 63) / 64 * 64;
  *len = static_cast<int>(L);
  *n = static_cast<int>((c.N + L - 1) / L);
}

int64_t total_segments(const LinCall& c, int len, int n) {
  return c.T > 0 ? c.T / len + c.S : static_cast<int64_t>(c.S) * n;
}

}  // namespace

size_t lin_ws_bytes(const LinCall& c) {
  int len, n;
  segments(c, &len, &n);
  if (n == 1) return 0;
  const size_t rows = static_cast<size_t>(total_segments(c, len, n)) * c.H;
  return rows * sizeof(float) * c.dk * c.dv + ((rows * sizeof(float) + 255) & ~size_t(255));
}

hipError_t launch_linear_step(const LinCall& c, hipStream_t st) {
  const LinArgs a = lin_args(c);
  if (c.in_dt == RN_F32)
    return c.out_dt == RN_F32 ? launch_step_t<RN_F32, RN_F32>(a, st) : launch_step_t<RN_F32, RN_BF16>(a, st);
  return c.out_dt == RN_F32 ? launch_step_t<RN_BF16, RN_F32>(a, st) : launch_step_t<RN_BF16, RN_BF16>(a, st);
}

hipError_t launch_linear_chunked(const LinCall& c, hipStream_t st) {
  LinArgs a = lin_args(c);
  segments(c, &a.seg_len, &a.n_seg);
  const bool mfma = mfma_call(c);
  if (a.n_seg == 1) return mfma ? launch_lin_mfma(a, kLinWhole, st) : launch_recurrent<kLinWhole>(a, c.in_dt, c.out_dt, st);
  // Where N says little about the lengths: 1024 packed sequences of 28 tokens, 8 heads of 64 x 128,
  // and no nearer bound than the tokens of all: 216 us, 1382 us with S n_seg blocks (160 where the
  // bound is given, in one pass). (S N is then more than T, and T / L at most 768 by the choice of L.)
  a.flat = c.T > 0 && static_cast<int64_t>(c.S) * a.n_seg > 2 * (c.T / a.seg_len + c.S + 1);
  const size_t rows = static_cast<size_t>(total_segments(c, a.seg_len, a.n_seg)) * c.H;
  a.seg_decay = static_cast<float*>(c.ws);
  a.seg_state = a.seg_decay + ((rows + 63) & ~size_t(63));
  hipError_t e = mfma ? launch_lin_mfma(a, kLinState, st) : launch_recurrent<kLinState>(a, c.in_dt, c.out_dt, st);
  if (e != hipSuccess) return e;
  const unsigned z = a.flat ? static_cast<unsigned>(std::max<int64_t>(1, c.T / a.seg_len)) : c.S;
  if (c.dk * c.dv % 4 == 0)   // (states are 16-byte aligned, here and in the caller's buffers)
    hipLaunchKernelGGL(lin_scan<4>, dim3((c.dk * c.dv + 1023) / 1024, c.H, z), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(lin_scan<1>, dim3((c.dk * c.dv + 255) / 256, c.H, z), dim3(256), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.flat) return mfma ? launch_lin_mfma(a, kLinWhole, st) : launch_recurrent<kLinWhole>(a, c.in_dt, c.out_dt, st);
  return mfma ? launch_lin_mfma(a, kLinOut, st) : launch_recurrent<kLinOut>(a, c.in_dt, c.out_dt, st);
}

}  // namespace rn
