// Selective scan: what its kernels share.
//     D_t = softplus(dt_t + bias),  h_t = exp(D_t A) h_{t-1} + D_t x_t B_t,
//     y_t = C_t h_t + skip x_t,     out_t = y_t z_t sigmoid(z_t)
// for every channel, with n states each; channels of a group share B and C.
// Lanes are channels, so that B and C are the same for all lanes of a wave and come through scalar
// registers.
#pragma once
#include <type_traits>

#include "rn_kernels.h"
#include "sequences.h"

namespace rn {

constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f;   // log2(e) in two parts

struct ScanArgs {
  Seqs q;
  int32_t D, n, G, n_slots;
  int32_t tiles;                          // blocks along the channels of a group
  bool softplus, zero_rest;
  bool a4;                                // A's rows are whole fours on 16 bytes (states' always are, if whole)
  int64_t xs[2], dts[2], zs[2], os[2];    // sequence and token strides
  int64_t bs[3], cs[3];                   // sequence, group and token strides
  const int32_t* slots;
  const void* x;
  const void* dt;
  const void* z;
  const void* b;
  const void* c;
  const float* A;                         // [D][n]
  const float* skip;                      // [D] or null
  const float* bias;                      // [D] or null
  const float* state_in;
  float* state_out;
  void* out;
  float* seg_state;                       // [pieces][D][n]: what a segment adds, then its starting state
  float* seg_step;                        // [pieces][D]: the sum of a segment's D_t
};

// x log2(e), rounded once (the constant in two parts).
__device__ __forceinline__ float in_log2(float x) { return fmaf(x, kLog2eLow, x * kLog2e); }
// softplus(v) to float32 accuracy at any v, infinities too: max(v, 0) + log1p(e), e = exp(-|v|) (which is
// nothing beside 1 from |v| = 126 on, and beside v long before). What rounding the exponent loses goes back
// into e (it is |v| 2^-24 of it), and with w = 1 + e, what rounding w loses into the logarithm: log1p(e) =
// log(w) + (e - (w - 1)) / w, of which 1 / w is left out (the term is at most 2^-24 in all, and where w is
// not near 1 the result is not small). The hardware's logarithm is relative near 1.
__device__ __forceinline__ float softplus(float v) {
  const float m = -fminf(fabsf(v), 126.0f), t = m * kLog2e;
  float e = __builtin_amdgcn_exp2f(t);
  e = fmaf(e, fmaf(m, kLog2eLow, fmaf(m, kLog2e, -t)) * 0.6931472f, e);
  const float w = 1.0f + e;
  return (v < 0.0f ? 0.0f : v) + fmaf(__builtin_amdgcn_logf(w), 0.6931472f, e - (w - 1.0f));
}
// The exponent's rounding stays in here: with |v| 2^-24 (1 - sigmoid(v)) of the value it is 1e-6 where the value is
// 1e-9, while a step of that size, for which softplus puts it back, decides what a state keeps. (Three more of a
// token's and channel's 117 instructions.)
__device__ __forceinline__ float sigmoidf(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

template <int DT, class T>
__device__ __forceinline__ float value_of(T x) {
  if constexpr (DT == RN_F32) return x;
  else return bf16_to_f32(x);
}

// A channel's n states (or decays), zeros behind them; by fours where they are whole fours on 16 bytes.
template <int NS>
__device__ __forceinline__ void load_states(const float* p, int n, bool fours, float* v) {
  if (fours) {
#pragma unroll
    for (int i = 0; i < NS; i += 4) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) q = *reinterpret_cast<const float4*>(p + i);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
template <int NS>
__device__ __forceinline__ void store_states(float* p, int n, bool fours, const float* v) {
  if (fours) {
#pragma unroll
    for (int i = 0; i < NS; i += 4)
      if (i < n) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < n) p[i] = v[i];
  }
}

// The wave's first lane's value, as a scalar.
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(x) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// A lane's byte offset from uniform pointers for the accesses that follow, as the 32 bits that an access
// takes beside the scalar registers of its pointer. (Widened ahead of a loop, it would be added to every
// pointer by itself, in 64 bits.)
__device__ __forceinline__ unsigned lane_offset(unsigned bytes) {
  asm volatile("" : "+v"(bytes));
  return bytes;
}

// NS values of B or C from element i of p (both the same for the whole wave). FAST: through the scalar
// cache; all NS are there, bf16 in pairs that start on 4 bytes. Else every lane loads the first `have` of
// them, the rest being zeros.
template <int DT, int NS, bool FAST>
struct Uniform;
template <int DT, int NS>
struct Uniform<DT, NS, true> {
  static constexpr int kWords = DT == RN_F32 ? NS : NS / 2;
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const void* p, int64_t i, int) {
    typedef const __attribute__((address_space(4))) uint32_t* words;
    const words w = (words)static_cast<uint64_t>(uniform64(reinterpret_cast<int64_t>(p) + i * (DT == RN_F32 ? 4 : 2)));
#pragma unroll
    for (int k = 0; k < kWords; ++k) u[k] = w[k];
  }
  // What was unpacked so far is not kept: values are unpacked again when they are needed again.
  __device__ __forceinline__ void fresh() {
    if constexpr (DT != RN_F32) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) asm volatile("" : "+s"(u[k]));
    }
  }
  __device__ __forceinline__ float value(int k) const {
    if constexpr (DT == RN_F32) return __uint_as_float(u[k]);
    else return __uint_as_float(k % 2 ? u[k / 2] & 0xffff0000u : u[k / 2] << 16);
  }
};
template <int DT, int NS>
struct Uniform<DT, NS, false> {
  float f[NS];
  __device__ __forceinline__ void load(const void* p, int64_t i, int have) {
#pragma unroll
    for (int k = 0; k < NS; ++k) f[k] = k < have ? Elem<DT>::load(p, i + k) : 0.f;
  }
  __device__ __forceinline__ void fresh() {}
  __device__ __forceinline__ float value(int k) const { return f[k]; }
};

// Whether B and C can come through the scalar cache: all states in whole sets of `set`, in bf16 as pairs that start on
// 4 bytes. Elsewhere every lane loads them for itself into registers of its own, which costs 2 to 6 times the time
// (bf16 with gate, prompts of 8192 tokens x 2048 channels / gradients of 4 x 2048 x 1024: 16 states 138 / 247 us, with
// B and C 2 bytes off 406 / 815; 24 states 185 / 532 and 20 states 695 / 1114; 48 states 379 / 1875 and 40 states 2330 /
// 3430).
inline bool scan_fast(const ScanArgs& a, int dt, int set) {
  if (a.n % set) return false;
  if (dt == RN_F32) return true;
  for (int i = 0; i < 3; ++i)
    if (a.bs[i] % 2 || a.cs[i] % 2) return false;
  return reinterpret_cast<uintptr_t>(a.b) % 4 == 0 && reinterpret_cast<uintptr_t>(a.c) % 4 == 0;
}

// The call's kernel arguments, with `len` tokens a piece.
inline ScanArgs scan_args(const ScanCall& c, int len) {
  ScanArgs a;
  a.q = Seqs{c.S, c.N, c.T, 0, 0, c.cu, c.lens};
  seq_cut(&a.q, len);
  a.D = c.D; a.n = c.n; a.G = c.G; a.n_slots = c.n_slots; a.tiles = (c.D / c.G + 63) / 64;
  a.softplus = c.softplus; a.zero_rest = c.zero_rest;
  for (int i = 0; i < 2; ++i) { a.xs[i] = c.xs[i]; a.dts[i] = c.dts[i]; a.zs[i] = c.zs[i]; a.os[i] = c.os[i]; }
  for (int i = 0; i < 3; ++i) { a.bs[i] = c.bs[i]; a.cs[i] = c.cs[i]; }
  a.a4 = c.n % 4 == 0 && reinterpret_cast<uintptr_t>(c.A) % 16 == 0;
  a.slots = c.slots; a.x = c.x; a.dt = c.dt; a.z = c.z; a.b = c.b; a.c = c.c; a.A = c.A; a.skip = c.skip; a.bias = c.bias;
  a.state_in = c.state_in; a.state_out = c.state_out; a.out = c.out; a.seg_state = nullptr; a.seg_step = nullptr;
  return a;
}

}  // namespace rn
