// Linear attention with a decay per head and token, in float32:
//     S_t = exp(g_t) S_{t-1} + k_t^T v_t,     o_t = scale q_t S_t.
//
// lin_step: one token a sequence. Bound by HBM: the float32 state is read and written once.
// lin_float: prompts of any type and head size in chunks of 16 tokens on the float32 matrix cores
// (bf16 in and float32 out, 32 heads of 2048 tokens, 128 x 128: 129 us; bf16 of 100 x 100: 126 us).
// Bound by the wait for each chunk's phases and the padding of small heads (padded float32 batch of
// 3 sequences of up to 2001 tokens, 5 heads of 48 x 81: 32 us, of which the scan is 8; 32 heads of
// 2048 tokens, 128 x 128: 131 us). The recurrence itself, token by token on the vector units,
// took 39 and 172 us.
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
// no load hangs on a condition (128 states of 16 heads of 256 x 512: 355 us, 6.1 TB/s, where a
// program steps the same states, 380 to 390 on states in a pool's order; with conditions and half the
// columns a block 460 us. Of 256 x 384 in three slices of 128 columns: 289 us, with conditions 432; of
// 128 x 192 in three of 64: 67 and 98 us).
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

// ---- prompts in float32 -------------------------------------------------------------------
// Chunks of 16 tokens, with c_t the running sum of the log2 decays inside one:
//     O = (Q K^T o D) V + diag(2^c) Q S,  D_ts = 2^(c_t - c_s) for s <= t;
//     S <- 2^(c_15) S + K^T (w o V),  w_s = 2^(c_15 - c_s),
// all products on the float32 matrix cores. A block owns 64 columns of one head's state over one
// segment of one sequence; wave w has its rows [w RW, (w+1) RW) as accumulators (rows past d_k stay
// zero), which hold four rows of a column a lane: with the reduction's rows numbered 4 (l / 16) + r
// they are the operand of Q S as they are. Each wave forms its rows' shares of the scores and of
// Q S; the shares meet in LDS, and wave w finishes the columns [16 w, 16 w + 16).
constexpr int kTok = 16;
constexpr int kCols = 64;
constexpr int kPad = 4;      // floats behind each LDS row, so that 16 rows at a column, and 4 rows of
                             // 16 columns at a distance of 4 rows, lie in different banks

struct alignas(16) Decays16 {   // of one chunk
  double c[kTok];        // running sum of log2 decays
  float e[kTok];         // 2^c
  float w[kTok];         // 2^(c_15 - c)
  float a;               // 2^c_15
  int bad;               // v holds a NaN or an infinity
};

__device__ __forceinline__ f32x4 mfma32(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
template <int CTRL>
__device__ __forceinline__ double row_shifted(double x) {   // 0 where a row of 16 lanes has no such lane
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// One wave whose lanes l hold the log decay of token l % 16. Returns the sum of log2 decays. (A
// decay of 0 counts as 2^-173, which is 0 as a float32 factor.)
__device__ __forceinline__ double scan_decays16(float g, Decays16* d) {
  const int lane = threadIdx.x & 63;
  double x = static_cast<double>(g) * 1.4426950408889634;
  if (x < -173.0) x = -173.0;           // (a NaN stays)
  x += row_shifted<0x111>(x);
  x += row_shifted<0x112>(x);
  x += row_shifted<0x114>(x);
  x += row_shifted<0x118>(x);
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 15);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 15);
  const double last = __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
  if (lane < kTok) {
    d->c[lane] = x;
    d->e[lane] = __builtin_amdgcn_exp2f(static_cast<float>(x));
    d->w[lane] = __builtin_amdgcn_exp2f(static_cast<float>(last - x));
    if (lane == 15) d->a = __builtin_amdgcn_exp2f(static_cast<float>(x));
  }
  return last;
}

template <int IN, int OUT, int RW, LinMode MODE>
__global__ void __launch_bounds__(256) lin_float(LinArgs a) {
  constexpr int D = 4 * RW;
  constexpr int RT = RW / 16;             // 16-row tiles of the state a wave
  constexpr int CT = kCols / 16;          // 16-column tiles
  constexpr int E = kTok * D / 256;       // q (or k) elements a thread stages
  constexpr bool kOut = MODE != kLinState;
  __shared__ __align__(16) float qt[kOut ? kTok : 1][D + kPad];
  __shared__ __align__(16) float kt[kTok][D + kPad];
  __shared__ __align__(16) float vt[kTok][kCols + kPad];
  __shared__ __align__(16) float pt[kOut ? 4 : 1][kTok][kTok + kPad];       // the waves' shares of the scores
  __shared__ __align__(16) float part[kOut ? 4 : 1][kTok][kCols + kPad];    // and of Q S
  __shared__ Decays16 dec[2];
  int h, c0;
  lin_block(a, blockIdx.x, &h, &c0);
  c0 *= kCols;
  int seg, s;
  if (!lin_place(a, &s, &seg)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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

  const int l16 = lane & 15, g4 = (lane >> 4) * 4;
  f32x4 S[RT][CT];                        // rows wave RW + 16 i + g4 + r, column 16 c + l16
  {
    const float* from = MODE == kLinState ? nullptr
                        : MODE == kLinOut || !one ? a.seg_state + (lin_segment(a, s, row0, seg) * a.H + h) * sh
                        : a.state_in && slot >= 0 ? a.state_in + (static_cast<int64_t>(slot) * a.H + h) * sh : nullptr;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = wave * RW + 16 * i + g4 + r, v = 16 * c + l16;
          S[i][c][r] = from && d < a.dk && v < nc ? from[static_cast<int64_t>(d) * a.dv + c0 + v] : 0.f;
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
  };
  // (log decays are fetched two chunks ahead: one wave forms a chunk's decays during the one before)
  auto fetch_g = [&](int t) { rg = t + l16 < t1 ? a.g[go + (t + l16) * a.gs[2]] : 0.f; };
  double gsum = 0.0;
  if (t0 < t1) {
    fetch(t0);
    fetch_g(t0);
    if (wave == 3) gsum += scan_decays16(rg, &dec[0]);
    fetch_g(t0 + kTok);
    if (tid < 2) dec[tid].bad = 0;
    __syncthreads();
  }
  int buf = 0;
  for (int t = t0; t < t1; t += kTok, buf ^= 1) {
    const int n = min(kTok, t1 - t);
    // (tokens behind the last have decay 1 and k = q = v = 0, and change nothing)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = tid + 256 * e;
      const bool ok = i / D < n && i % D < a.dk;
      if constexpr (kOut) qt[i / D][i % D] = ok ? rq[e] : 0.f;
      kt[i / D][i % D] = ok ? rk[e] : 0.f;
    }
    bool mine = false;
#pragma unroll
    for (int e = 0; e < kTok * kCols / 256; ++e) {
      const int i = tid + 256 * e;
      const float x = i / kCols < n && i % kCols < nc ? rv[e] : 0.f;
      mine |= !(fabsf(x) < INFINITY);
      vt[i / kCols][i % kCols] = x;
    }
    if (kOut && mine) dec[buf].bad = 1;
    __syncthreads();
    if (t + kTok < t1) {
      fetch(t + kTok);
      if (wave == 3) gsum += scan_decays16(rg, &dec[buf ^ 1]);
      fetch_g(t + 2 * kTok);
    }
    const Decays16& Y = dec[buf];
    float vf[4];                          // tokens g4 + n of this wave's output columns
    if constexpr (kOut) {
#pragma unroll
      for (int n = 0; n < 4; ++n) vf[n] = vt[g4 + n][16 * wave + l16];
      f32x4 P = {}, O[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) O[c] = f32x4{};
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const f32x4 q = *reinterpret_cast<const f32x4*>(&qt[l16][wave * RW + 16 * i + g4]);
        const f32x4 k = *reinterpret_cast<const f32x4*>(&kt[l16][wave * RW + 16 * i + g4]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          P = mfma32(q[r], k[r], P);
#pragma unroll
          for (int c = 0; c < CT; ++c) O[c] = mfma32(q[r], S[i][c][r], O[c]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        pt[wave][g4 + r][l16] = P[r];
#pragma unroll
        for (int c = 0; c < CT; ++c) part[wave][g4 + r][16 * c + l16] = O[c][r];
      }
    }
    if (MODE != kLinOut || t + kTok < t1) {
      const float a16 = Y.a;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[i][c] *= a16;
      const f32x4 w = *reinterpret_cast<const f32x4*>(&Y.w[g4]);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float wv[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) wv[c] = w[n] * vt[g4 + n][16 * c + l16];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const float k = kt[g4 + n][wave * RW + 16 * i + l16];
#pragma unroll
          for (int c = 0; c < CT; ++c) S[i][c] = mfma32(k, wv[c], S[i][c]);
        }
      }
    }
    if (tid == 0) dec[buf ^ 1].bad = 0;
    // The shares are whole, and the tiles of Q, K and V are free (but see `bad`).
    __syncthreads();
    if constexpr (kOut) {
      const f32x4 e = *reinterpret_cast<const f32x4*>(&Y.e[g4]);
      f32x4 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float* x = &part[0][g4 + r][16 * wave + l16];
        constexpr int W = kTok * (kCols + kPad);
        o[r] = e[r] * ((x[0] + x[W]) + (x[2 * W] + x[3 * W]));
      }
      const bool bad = __builtin_amdgcn_readfirstlane(Y.bad);   // (one for the block)
      if (bad)
#pragma unroll
        for (int n = 0; n < 4; ++n) vf[n] = fabsf(vf[n]) < INFINITY ? vf[n] : 0.f;
      f32x4 p = *reinterpret_cast<const f32x4*>(&pt[0][l16][g4]);
#pragma unroll
      for (int w = 1; w < 4; ++w) p += *reinterpret_cast<const f32x4*>(&pt[w][l16][g4]);
      const double cq = Y.c[l16];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float x = p[n] * __builtin_amdgcn_exp2f(static_cast<float>(cq - Y.c[g4 + n]));
        o = mfma32(g4 + n <= l16 ? x : 0.f, vf[n], o);
      }
      if (bad) {
        // 0 times a NaN or an infinity of a later token must not reach this one: what was left out
        // of the product, for the queries that see it
#pragma unroll 1
        for (int k = 0; k < g4 + 4; ++k) {
          const float v = vt[k][16 * wave + l16];
          if (!(fabsf(v) < INFINITY)) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int q = g4 + r;
              const float x = (pt[0][q][k] + pt[1][q][k] + pt[2][q][k] + pt[3][q][k]) * __builtin_amdgcn_exp2f(static_cast<float>(Y.c[q] - Y.c[k]));
              o[r] = k <= q ? fmaf(x, v, o[r]) : o[r];
            }
          }
        }
        __syncthreads();
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (g4 + r < n && 16 * wave + l16 < nc)
          Elem<OUT>::store(a.out, oo + (t + g4 + r) * a.os[2] + 16 * wave + l16, a.scale * o[r]);
    }
  }
  float* to = nullptr;
  if (MODE == kLinWhole && keep && one) to = a.state_out + (static_cast<int64_t>(slot) * a.H + h) * sh;
  if (MODE == kLinState) {
    const int64_t i = lin_segment(a, s, row0, seg) * a.H + h;
    to = a.seg_state + i * sh;
    if (c0 == 0 && tid == 192) a.seg_decay[i] = __builtin_amdgcn_exp2f(static_cast<float>(gsum));
  }
  if (to) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = wave * RW + 16 * i + g4 + r, v = 16 * c + l16;
          if (d < a.dk && v < nc) to[static_cast<int64_t>(d) * a.dv + c0 + v] = S[i][c][r];
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
hipError_t launch_float_t(const LinArgs& a, hipStream_t st) {
  const int slices = (a.dv + kCols - 1) / kCols;
  const bool rest = a.T > 0 && a.zero_rest && MODE != kLinState;
  const dim3 grid = lin_grid(a, a.H * slices, rest);
  const int rw = (a.dk + 3) / 4;
  if (rw <= 16) hipLaunchKernelGGL((lin_float<IN, OUT, 16, MODE>), grid, dim3(256), 0, st, a);
  else if (rw <= 32) hipLaunchKernelGGL((lin_float<IN, OUT, 32, MODE>), grid, dim3(256), 0, st, a);
  else if (rw <= 48) hipLaunchKernelGGL((lin_float<IN, OUT, 48, MODE>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((lin_float<IN, OUT, 64, MODE>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <LinMode MODE>
hipError_t launch_float(const LinArgs& a, int in_dt, int out_dt, hipStream_t st) {
  if (in_dt == RN_F32)
    return out_dt == RN_F32 ? launch_float_t<RN_F32, RN_F32, MODE>(a, st) : launch_float_t<RN_F32, RN_BF16, MODE>(a, st);
  return out_dt == RN_F32 ? launch_float_t<RN_BF16, RN_F32, MODE>(a, st) : launch_float_t<RN_BF16, RN_BF16, MODE>(a, st);
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
    if (states >= 512) {      // the widest slices of whole columns that whole batches of rows go with
      if (a.dv % 512 == 0 && a.dk % 32 == 0) RN_STEP(4, 128, 512, true);
      if (a.dv % 256 == 0 && a.dk % 64 == 0) RN_STEP(4, 64, 512, true);
      if (a.dv % 128 == 0 && a.dk % 64 == 0) RN_STEP(4, 32, 256, true);
      if (a.dv % 64 == 0 && a.dk % 128 == 0) RN_STEP(4, 16, 256, true);
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
// not known when the workspace is sized: a call with an unaligned one takes the float32
// kernel on the same segments.)
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
// sequence of less than three segments stays whole. (In float32, segments of
// 32 tokens: 8 heads of 300, 64 x 64, 24 -> 21 us, but of 2000 32 -> 40.)
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

// Blocks along the segments of all sequences, where N says little about the lengths: 1024 packed
// sequences of 28 tokens, 8 heads of 64 x 128, and no nearer bound than the tokens of all: 233 us,
// 1622 us with S n_seg blocks (175 where the bound is given, in one pass). (S N is then more than T,
// and T / L at most 768 by the choice of L.)
bool flat_grid(const LinCall& c, int len, int n) {
  return n > 1 && c.T > 0 && static_cast<int64_t>(c.S) * n > 2 * (c.T / len + c.S + 1);
}

// Segment states in the workspace (lin_segment()). In a packed batch they grow with the tokens, not
// with S or with T alone: S n is at most 2 (T / L + S + 1) where the grid is not flat, and n is at
// least three.
int64_t total_segments(const LinCall& c, int len, int n) {
  return flat_grid(c, len, n) ? 2 * c.T / len : static_cast<int64_t>(c.S) * n;
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
  if (a.n_seg == 1) return mfma ? launch_lin_mfma(a, kLinWhole, st) : launch_float<kLinWhole>(a, c.in_dt, c.out_dt, st);
  a.flat = flat_grid(c, a.seg_len, a.n_seg);
  const size_t rows = static_cast<size_t>(total_segments(c, a.seg_len, a.n_seg)) * c.H;
  a.seg_decay = static_cast<float*>(c.ws);
  a.seg_state = a.seg_decay + ((rows + 63) & ~size_t(63));
  hipError_t e = mfma ? launch_lin_mfma(a, kLinState, st) : launch_float<kLinState>(a, c.in_dt, c.out_dt, st);
  if (e != hipSuccess) return e;
  const unsigned z = a.flat ? static_cast<unsigned>(std::max<int64_t>(1, c.T / a.seg_len)) : c.S;
  if (c.dk * c.dv % 4 == 0)   // (states are 16-byte aligned, here and in the caller's buffers)
    hipLaunchKernelGGL(lin_scan<4>, dim3((c.dk * c.dv + 1023) / 1024, c.H, z), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(lin_scan<1>, dim3((c.dk * c.dv + 255) / 256, c.H, z), dim3(256), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.flat) return mfma ? launch_lin_mfma(a, kLinWhole, st) : launch_float<kLinWhole>(a, c.in_dt, c.out_dt, st);
  return mfma ? launch_lin_mfma(a, kLinOut, st) : launch_float<kLinOut>(a, c.in_dt, c.out_dt, st);
}

}  // namespace rn
