// Rows of d values in registers, as the norms hold them: pieces of a row, their loads and stores, and
// sums over the lanes and waves that share a row.
#pragma once
#include <type_traits>

#include "rn_device.h"

namespace rn {
namespace {

// Threads of a block whose rows take W waves each (0: 16 lanes), and lanes of a row.
constexpr int threads(int W) { return W > 4 ? 64 * W : 256; }
constexpr int lanes(int W) { return W ? 64 * W : 16; }

// How a row falls into pieces of V elements: every lane has all its pieces; some have none; or rows
// start anywhere and the last piece may be short. Memory takes 16-byte accesses at any element's
// address, so the last kind differs only in that piece (backward of 3001 x 1537 float32: 22 us, element
// by element 27; of 2000 x 10001 bf16: 75 and 216 us; forward 44 and 77).
enum Fit : int { kFull, kSome, kOdd };

// 16 or 8 bytes, past the caches with STREAM (which pays for calls larger than the last-level
// cache; what a smaller call leaves behind is soon read again).
template <bool STREAM, class T>
__device__ __forceinline__ T get(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const T*>(p));
  else return *static_cast<const T*>(p);
}
template <bool STREAM, class T>
__device__ __forceinline__ void put(void* p, const T& x) {
  if constexpr (STREAM) __builtin_nontemporal_store(x, static_cast<T*>(p));
  else *static_cast<T*>(p) = x;
}
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// the same at any address of a 16-bit element
typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(2)));

// V consecutive elements of type DT as they are in memory; an address of 16 bytes (or the whole,
// where that is less) but for kOdd. `left`: elements of the row from here on (kOdd).
template <int DT, int V, Fit FIT, bool STREAM = false>
struct Raw {
  static constexpr int kElem = DT == RN_F32 ? 4 : 2;
  static constexpr int kBytes = V * kElem;
  using T4 = typename std::conditional<FIT == kOdd, u32x4a, u32x4>::type;
  using T2 = typename std::conditional<FIT == kOdd, u32x2a, u32x2>::type;
  uint32_t u[kBytes / 4];
  __device__ __forceinline__ void load(const void* p, int64_t i, int left) {
    const char* s = static_cast<const char*>(p) + i * kElem;
    if (FIT == kOdd && left < V) {
      clear();
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < left) {
          if constexpr (DT == RN_F32) u[j] = *reinterpret_cast<const uint32_t*>(s + 4 * j);
          else u[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(s + 2 * j)) << (j % 2 * 16);
        }
    } else if constexpr (kBytes >= 16) {
#pragma unroll
      for (int j = 0; j < kBytes / 16; ++j) {
        const T4 x = get<STREAM, T4>(s + 16 * j);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[4 * j + k] = x[k];
      }
    } else {
      const T2 x = get<STREAM, T2>(s);
      u[0] = x[0]; u[1] = x[1];
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i, int left) const {
    char* s = static_cast<char*>(p) + i * kElem;
    if (FIT == kOdd && left < V) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j < left) {
          if constexpr (DT == RN_F32) *reinterpret_cast<uint32_t*>(s + 4 * j) = u[j];
          else *reinterpret_cast<uint16_t*>(s + 2 * j) = static_cast<uint16_t>(u[j / 2] >> (j % 2 * 16));
        }
    } else if constexpr (kBytes >= 16) {
#pragma unroll
      for (int j = 0; j < kBytes / 16; ++j) put<STREAM>(s + 16 * j, T4{u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]});
    } else {
      put<STREAM>(s, T2{u[0], u[1]});
    }
  }
  __device__ __forceinline__ float value(int j) const {
    if constexpr (DT == RN_F32) return __uint_as_float(u[j]);
    else return j % 2 ? __uint_as_float(u[j / 2] & 0xffff0000u) : __uint_as_float(u[j / 2] << 16);
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (DT == RN_F32) {
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] = __float_as_uint(f[j]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) u[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < kBytes / 4; ++j) u[j] = 0;
  }
};
template <int DT, int V, Fit FIT, bool STREAM = false>
__device__ __forceinline__ void load(const void* p, int64_t i, int left, float* f) {
  Raw<DT, V, FIT, STREAM> r;
  r.load(p, i, left);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = r.value(j);
}
template <int DT, int V, Fit FIT, bool STREAM = false>
__device__ __forceinline__ void store(void* p, int64_t i, int left, const float* f) {
  Raw<DT, V, FIT, STREAM> r;
  r.set(f);
  r.store(p, i, left);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_zero(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, true));
}
// Sum over a wave, in every lane: over the 16 lanes of each row, over the rows, from lane 63.
__device__ __forceinline__ float wave_total(float x) {
  x += dpp_or_zero<0x111, 0xf>(x);
  x += dpp_or_zero<0x112, 0xf>(x);
  x += dpp_or_zero<0x114, 0xf>(x);
  x += dpp_or_zero<0x118, 0xf>(x);
  x += dpp_or_zero<0x142, 0xa>(x);
  x += dpp_or_zero<0x143, 0xc>(x);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Sum over the 16 lanes of each row of a wave, in all of them.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_total(float x) {
  x += dpp<0xB1>(x);                      // lane ^ 1
  x += dpp<0x4E>(x);                      // lane ^ 2
  x += dpp<0x141>(x);                     // lane i <-> 7 - i within 8
  return x + dpp<0x140>(x);               // lane i <-> 15 - i
}

// Sums of N values over the W waves that share a row; every thread receives them. `red` holds
// W N floats. The caller does not write the same area again before a barrier has passed since.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float* red) {
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = W ? wave_total(x[n]) : row_total(x[n]);
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[w * N + n] = x[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      x[n] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) x[n] += red[i * N + n];
    }
  }
}

}  // namespace
}  // namespace rn
