// Layer norm of rows of d values, forward (with the residual sum) and backward (with the
// weight's and bias's gradients).
//
// Forward, per row: h = x + r; mean; then the biased variance of h - mean; y = (h - mean)
// rstd w + b. Backward, with g = dy w and xh = (x - mean) rstd: dx = rstd (g - mean(g) -
// xh mean(g xh)) + dh, dw = sum_rows dy xh, db = sum_rows dy.
//
// Bound by HBM: every tensor is read or written once (16384 x 4096 bf16: forward with residual
// 96 us, 5.6 TB/s; backward with the residual's gradient 108 us, 5.0 TB/s; a large copy reaches
// 4.9 to 5.4 TB/s on the card). Smaller calls are bound by latency (backward of 3001 x 1537
// float32: 22 us, of which the reduction of the weights' sums is 5). A row lives in the registers of 16
// lanes (W = 0, 16 rows per 256-thread block), of one wave (W = 1) or of a whole block (W = 4 or
// 16), so the passes
// over it (mean, centred squares, result) cost no memory access. Blocks walk over rows:
// the weights, and in the backward the column sums of dw and db, then stay in registers
// too, and the backward writes one partial row of sums per block, which a second kernel
// adds in a fixed order.
#include <algorithm>
#include <type_traits>

#include "rn_device.h"
#include "rn_kernels.h"

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

struct NormArgs {
  int64_t rows;
  int32_t d;
  float eps, fd;              // fd: d
  int64_t xs, rs, ss, os;   // row strides: x, residual / dsum, sum_out / dx, out / dout
  const void* x;
  const void* r;            // residual / dsum or null
  const float* w;
  const float* b;
  void* sum;                // sum_out or null / dx
  void* out;                // out
  const void* dout;
  float* part;              // partial sums of the backward: [blocks][2][d] or null
};

// Thread `lane` of a row's L lanes holds elements [V (lane + L i), +V) for i < NV.
template <int IN, int OUT, int V, int W, int NV, Fit FIT, bool STREAM>
__global__ void __launch_bounds__(threads(W)) norm_rows(NormArgs a) {
  constexpr int L = lanes(W);
  constexpr int R = threads(W) / L;       // rows per block
  __shared__ float red[2][W ? W : 1];
  const int lane = threadIdx.x % L;
  float w[NV * V], b[NV * V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = V * (lane + L * i);
#pragma unroll
    for (int j = 0; j < V; ++j) { w[i * V + j] = 1.f; b[i * V + j] = 0.f; }
    if (FIT == kFull || c < a.d) {
      if (a.w) load<RN_F32, V, FIT>(a.w, c, a.d - c, w + i * V);
      if (a.b) load<RN_F32, V, FIT>(a.b, c, a.d - c, b + i * V);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / L; row < a.rows; row += step) {
    float h[NV * V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
#pragma unroll
      for (int j = 0; j < V; ++j) h[i * V + j] = 0.f;
      if (FIT == kFull || c < a.d) load<IN, V, FIT, STREAM>(a.x, row * a.xs + c, a.d - c, h + i * V);
    }
    if (a.r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = V * (lane + L * i);
        if (FIT == kFull || c < a.d) {
          float t[V];
          load<IN, V, FIT, STREAM>(a.r, row * a.rs + c, a.d - c, t);
#pragma unroll
          for (int j = 0; j < V; ++j) h[i * V + j] += t[j];
        }
      }
    }
    if (a.sum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = V * (lane + L * i);
        if (FIT == kFull || c < a.d) store<IN, V, FIT, STREAM>(a.sum, row * a.ss + c, a.d - c, h + i * V);
      }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV * V; ++i) s[0] += h[i];
    row_sums<W>(s, red[0]);
    const float mean = s[0] / a.fd;
    float s2[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[i * V + j] -= mean;
        if (FIT == kFull || V * (lane + L * i) + (FIT == kOdd ? j : 0) < a.d) s2[0] = fmaf(h[i * V + j], h[i * V + j], s2[0]);
      }
    row_sums<W>(s2, red[1]);
    const float rstd = 1.0f / sqrtf(s2[0] / a.fd + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (FIT == kFull || c < a.d) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = fmaf(h[i * V + j] * rstd, w[i * V + j], b[i * V + j]);
        store<OUT, V, FIT, STREAM>(a.out, row * a.os + c, a.d - c, y);
      }
    }
  }
}

// With c = x - mean: the sums of c c, g and g c after the mean are all a row needs (mean(g xh)
// is rstd mean(g c)), so a row takes two joins of the block. The next row's values are on
// their way while a row is worked on.
template <int IN, int OUT, int V, int W, int NV, Fit FIT, bool STREAM>
__global__ void __launch_bounds__(threads(W)) norm_rows_backward(NormArgs a) {
  constexpr int L = lanes(W);
  constexpr int R = threads(W) / L;
  constexpr bool kAhead = W < 16 || NV * V <= 4;   // blocks of 16 waves have 128 registers a lane
  __shared__ float red[2][W ? 4 * W : 1];         // rows take the areas in turn
  __shared__ float merge[W <= 1 ? L * NV * V : 1];
  const int lane = threadIdx.x % L;
  float dw[NV * V], db[NV * V];
#pragma unroll
  for (int i = 0; i < NV * V; ++i) { dw[i] = 0.f; db[i] = 0.f; }
  Raw<IN, V, FIT, STREAM> rx[NV], rr[NV];
  Raw<OUT, V, FIT, STREAM> rg[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (FIT == kFull || c < a.d) {
        rx[i].load(a.x, row * a.xs + c, a.d - c);
        rg[i].load(a.dout, row * a.os + c, a.d - c);
        if (a.r) rr[i].load(a.r, row * a.rs + c, a.d - c);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) { rx[i].clear(); rg[i].clear(); rr[i].clear(); }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / L;
  if (kAhead && row < a.rows) fetch(row);
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    if (!kAhead) fetch(row);
    float x[NV * V], g[NV * V], t[NV * V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[i * V + j] = rx[i].value(j);
        g[i * V + j] = rg[i].value(j);
        t[i * V + j] = rr[i].value(j);
        s[0] += x[i * V + j];
      }
    if (kAhead && row + step < a.rows) fetch(row + step);
    row_sums<W>(s, red[turn]);
    const float mean = s[0] / a.fd;
    float m[3] = {0.f, 0.f, 0.f};         // sums of c c, g w, g w c
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (FIT == kFull || c < a.d) {
        float wt[V];
#pragma unroll
        for (int j = 0; j < V; ++j) wt[j] = 1.f;
        if (a.w) load<RN_F32, V, FIT>(a.w, c, a.d - c, wt);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = i * V + j;
          x[e] = FIT != kOdd || c + j < a.d ? x[e] - mean : 0.f;
          db[e] += g[e];
          const float gw = g[e] * wt[j];
          m[0] = fmaf(x[e], x[e], m[0]);
          m[1] += gw;
          m[2] = fmaf(gw, x[e], m[2]);
        }
      }
    }
    row_sums<W>(m, red[turn] + W);
    const float rstd = 1.0f / sqrtf(m[0] / a.fd + a.eps);
    const float sg = m[1] / a.fd, sgx = m[2] / a.fd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (FIT == kFull || c < a.d) {
        float wt[V];
#pragma unroll
        for (int j = 0; j < V; ++j) wt[j] = 1.f;
        if (a.w) load<RN_F32, V, FIT>(a.w, c, a.d - c, wt);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = i * V + j;
          const float xh = x[e] * rstd;
          dw[e] = fmaf(g[e], xh, dw[e]);
          t[e] = fmaf(rstd, g[e] * wt[j] - sg - xh * sgx, t[e]);
        }
        store<IN, V, FIT, STREAM>(a.sum, row * a.ss + c, a.d - c, t + i * V);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.d;
  if constexpr (W <= 1) {
    // the sums of a wave's rows, then of the four waves, added in their order
    if constexpr (W == 0) {
#pragma unroll
      for (int i = 0; i < NV * V; ++i) {
        dw[i] += __shfl_xor(dw[i], 16); dw[i] += __shfl_xor(dw[i], 32);
        db[i] += __shfl_xor(db[i], 16); db[i] += __shfl_xor(db[i], 32);
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* v = which ? db : dw;
      for (int wv = 0; wv < 4; ++wv) {
        if (static_cast<int>(threadIdx.x >> 6) == wv && (threadIdx.x & 63) < L) {
#pragma unroll
          for (int i = 0; i < NV * V; ++i) {
            float* m = &merge[i * L + lane];
            *m = wv == 0 ? v[i] : *m + v[i];
          }
        }
        __syncthreads();
      }
      if (threadIdx.x < L) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = V * (lane + L * i);
          if (FIT == kFull || c < a.d) {
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (FIT != kOdd || c + j < a.d) part[static_cast<int64_t>(which) * a.d + c + j] = merge[(i * V + j) * L + lane];
          }
        }
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (FIT == kFull || c < a.d) {
        store<RN_F32, V, FIT>(part, c, a.d - c, dw + i * V);
        store<RN_F32, V, FIT>(part + a.d, c, a.d - c, db + i * V);
      }
    }
  }
}

// dweight and dbias: the partial rows added in the order of their blocks, 32 interleaved sums
// a column which are then added in turn. One block takes 32 columns of the 2 d.
__global__ void __launch_bounds__(1024) norm_reduce(const float* part, int blocks, int d, float* dw, float* db) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  const int grp = threadIdx.x >> 5;
  float s = 0.f;
  if (col < 2 * d) {
#pragma unroll 8
    for (int i = grp; i < blocks; i += 32) s += part[static_cast<int64_t>(i) * 2 * d + col];
  }
  red[grp][threadIdx.x & 31] = s;
  __syncthreads();
  if (grp == 0 && col < 2 * d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    float* out = col < d ? dw : db;
    if (out) out[col < d ? col : col - d] = s;
  }
}

// Rows that 16 lanes hold in two pieces each: four rows a wave (262144 x 128 bf16: forward 42 us,
// backward 44; with a wave a row 80 and 135).
bool narrow(const NormCall& n) { return n.d <= 32 * (n.in_dt == RN_BF16 ? 8 : 4); }

int backward_blocks(const NormCall& n) {
  // Three blocks a CU, which is what registers allow (rows of 16 waves: one), and at least four rows a
  // block (16 narrow ones, which it takes at a time). A block leaves 2 d floats of partial sums, written
  // and read once: with four rows that is half as much again as bf16 tensors with a residual, but
  // fewer blocks leave the chip empty (bf16 rows of 4096 with residual, at least 2, 4 or 8 rows a block:
  // 1024 rows 19, 17 and 21 us, 2048 rows 24, 23 and 23; 2048 rows of 12288 72, 59 and 50; 3001 x 1537
  // float32 24, 25 and 28).
  const int rows = narrow(n) ? 16 : 4;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((n.rows + rows - 1) / rows, 768)));
}

template <int IN, int OUT, int V, int W, int NV, Fit FIT, bool STREAM>
hipError_t launch_full(const NormCall& n, NormArgs a, hipStream_t st) {
  if (!n.backward) {
    constexpr int R = threads(W) / lanes(W);
    const int64_t need = (n.rows + R - 1) / R;
    hipLaunchKernelGGL((norm_rows<IN, OUT, V, W, NV, FIT, STREAM>), dim3(static_cast<unsigned>(std::min<int64_t>(need, 2048))),
                       dim3(threads(W)), 0, st, a);
    return hipGetLastError();
  }
  const int blocks = backward_blocks(n);
  hipLaunchKernelGGL((norm_rows_backward<IN, OUT, V, W, NV, FIT, STREAM>), dim3(blocks), dim3(threads(W)), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.part) {
    hipLaunchKernelGGL(norm_reduce, dim3((2 * n.d + 31) / 32), dim3(1024), 0, st, a.part, blocks, n.d, n.dw, n.db);
    e = hipGetLastError();
  }
  return e;
}

template <int IN, int OUT, int V, int W, int NV>
hipError_t launch_one(const NormCall& n, const NormArgs& a, hipStream_t st) {
  // Past the caches: the call's bytes against the 256 MB last-level cache (16384 x 4096 bf16 with
  // residual: 96 us past the caches, 103 us through them, backward 108 and 114; 16384 x 6144 138 and 148,
  // 185 and 193; 16384 x 4001 114 and 119, 171 and 175). Not where short rows share their 64-byte lines,
  // which would then be fetched for each (300000 x 200 bf16: 125 and 112, 124 and 116).
  const int64_t bytes = n.rows * n.d * ((IN == RN_F32 ? 4 : 2) * (n.r ? 2 : 1) + (OUT == RN_F32 ? 4 : 2) + (n.sum ? (IN == RN_F32 ? 4 : 2) : 0));
  const int64_t row = static_cast<int64_t>(n.d) * (IN == RN_F32 ? 4 : 2);
  const bool stream = bytes > (int64_t(256) << 20) && (row % 64 == 0 || row >= 2048);
  if (!n.vec) return stream ? launch_full<IN, OUT, V, W, NV, kOdd, true>(n, a, st) : launch_full<IN, OUT, V, W, NV, kOdd, false>(n, a, st);
  if (n.d != V * lanes(W) * NV)
    return stream ? launch_full<IN, OUT, V, W, NV, kSome, true>(n, a, st) : launch_full<IN, OUT, V, W, NV, kSome, false>(n, a, st);
  return stream ? launch_full<IN, OUT, V, W, NV, kFull, true>(n, a, st) : launch_full<IN, OUT, V, W, NV, kFull, false>(n, a, st);
}

template <int IN, int OUT>
hipError_t launch_t(const NormCall& n, const NormArgs& a, hipStream_t st) {
  // Waves a row and vectors a lane: at most 16 values of each tensor a lane, so that two rows
  // (one worked on, one on its way) and the sums over rows fit in its registers.
  constexpr int V = IN == RN_BF16 ? 8 : 4;   // 16 bytes of the input type
  const int nv = ((n.d + V - 1) / V + 63) / 64;      // vectors a lane of one wave
  if (narrow(n)) return n.d <= 16 * V ? launch_one<IN, OUT, V, 0, 1>(n, a, st) : launch_one<IN, OUT, V, 0, 2>(n, a, st);
  if (nv <= 1) return launch_one<IN, OUT, V, 1, 1>(n, a, st);
  if (nv <= 2) return launch_one<IN, OUT, V, 1, 2>(n, a, st);
  if (nv <= 4) return launch_one<IN, OUT, V, 4, 1>(n, a, st);
  if (nv <= 8) return launch_one<IN, OUT, V, 4, 2>(n, a, st);
  if constexpr (V == 8) {
    if (nv <= 16) return launch_one<IN, OUT, V, 16, 1>(n, a, st);
    return launch_one<IN, OUT, V, 16, 2>(n, a, st);
  } else {
    if (nv <= 16) return launch_one<IN, OUT, V, 4, 4>(n, a, st);
    if (nv <= 32) return launch_one<IN, OUT, V, 16, 2>(n, a, st);
    return launch_one<IN, OUT, V, 16, 4>(n, a, st);
  }
}

}  // namespace

size_t norm_backward_ws_bytes(const NormCall& n) {
  return static_cast<size_t>(backward_blocks(n)) * 2 * n.d * sizeof(float);
}

hipError_t launch_layernorm(const NormCall& n, hipStream_t st) {
  NormArgs a;
  a.rows = n.rows; a.d = n.d; a.eps = n.eps; a.fd = static_cast<float>(n.d);
  a.xs = n.xs; a.rs = n.rs; a.ss = n.ss; a.os = n.os;
  a.x = n.x; a.r = n.r; a.w = n.w; a.b = n.b; a.sum = n.sum; a.out = n.out; a.dout = n.dout;
  a.part = n.dw || n.db ? static_cast<float*>(n.ws) : nullptr;
  if (n.in_dt == RN_F32)
    return n.out_dt == RN_F32 ? launch_t<RN_F32, RN_F32>(n, a, st) : launch_t<RN_F32, RN_BF16>(n, a, st);
  return n.out_dt == RN_F32 ? launch_t<RN_BF16, RN_F32>(n, a, st) : launch_t<RN_BF16, RN_BF16>(n, a, st);
}

}  // namespace rn
