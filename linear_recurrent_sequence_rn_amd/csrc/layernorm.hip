// Layer norm of rows of d values, forward (with the residual sum) and backward (with the
// weight's and bias's gradients).
//
// Forward, per row: h = x + r; mean; then the biased variance of h - mean; y = (h - mean)
// rstd w + b. Backward, with g = dy w and xh = (x - mean) rstd: dx = rstd (g - mean(g) -
// xh mean(g xh)) + dh, dw = sum_rows dy xh, db = sum_rows dy.
//
// Bound by HBM: every tensor is read or written once. A row lives in the registers of one
// wave (W = 1, four rows per 256-thread block) or of a whole block (W = 4), so the passes
// over it (mean, centred squares, result) cost no memory access. Blocks walk over rows:
// the weights, and in the backward the column sums of dw and db, then stay in registers
// too, and the backward writes one partial row of sums per block, which a second kernel
// adds in a fixed order.
#include <algorithm>

#include "rn_device.h"
#include "rn_kernels.h"

namespace rn {
namespace {

constexpr int kThreads = 256;

// V consecutive elements of type DT from a 16-byte (V > 1) or element-aligned address.
template <int DT, int V> struct Vec;
template <> struct Vec<RN_F32, 1> {
  __device__ static __forceinline__ void load(const void* p, int64_t i, float* f) { f[0] = static_cast<const float*>(p)[i]; }
  __device__ static __forceinline__ void store(void* p, int64_t i, const float* f) { static_cast<float*>(p)[i] = f[0]; }
};
template <> struct Vec<RN_BF16, 1> {
  __device__ static __forceinline__ void load(const void* p, int64_t i, float* f) { f[0] = Elem<RN_BF16>::load(p, i); }
  __device__ static __forceinline__ void store(void* p, int64_t i, const float* f) { Elem<RN_BF16>::store(p, i, f[0]); }
};
template <int V> struct Vec<RN_F32, V> {
  __device__ static __forceinline__ void load(const void* p, int64_t i, float* f) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const float4 x = s[j];
      f[4 * j] = x.x; f[4 * j + 1] = x.y; f[4 * j + 2] = x.z; f[4 * j + 3] = x.w;
    }
  }
  __device__ static __forceinline__ void store(void* p, int64_t i, const float* f) {
    float4* s = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) s[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
  }
};
template <int V> struct Vec<RN_BF16, V> {   // V = 4 or 8
  __device__ static __forceinline__ void load(const void* p, int64_t i, float* f) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + i);
    uint32_t u[V / 2];
    if constexpr (V == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(s);
      u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(s);
      u[0] = x.x; u[1] = x.y;
    }
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      f[2 * j] = __uint_as_float(u[j] << 16);
      f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ void store(void* p, int64_t i, const float* f) {
    uint32_t u[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) u[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    uint16_t* s = static_cast<uint16_t*>(p) + i;
    if constexpr (V == 8) *reinterpret_cast<uint4*>(s) = make_uint4(u[0], u[1], u[2], u[3]);
    else *reinterpret_cast<uint2*>(s) = make_uint2(u[0], u[1]);
  }
};

// Sum of two values over the W waves that share a row; every thread receives both. `red`
// holds 2 W floats per use; callers alternate between two areas, so that one barrier per
// sum is enough.
template <int W>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    a += __shfl_xor(a, o, 64);
    b += __shfl_xor(b, o, 64);
  }
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) { red[2 * w] = a; red[2 * w + 1] = b; }
    __syncthreads();
    a = 0.f; b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) { a += red[2 * i]; b += red[2 * i + 1]; }
  }
}
template <int W>
__device__ __forceinline__ float row_sum(float a, float* red) {
  a = wave_sum(a);
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[w] = a;
    __syncthreads();
    a = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) a += red[i];
  }
  return a;
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

// Thread `lane` of a row's 64 W lanes holds elements [V (lane + 64 W i), +V) for i < NV.
template <int IN, int OUT, int V, int W, int NV>
__global__ void __launch_bounds__(kThreads) norm_rows(NormArgs a) {
  constexpr int L = 64 * W;
  constexpr int R = kThreads / L;         // rows per block
  constexpr bool kHold = NV * V <= 16;    // weights kept in registers
  __shared__ float red[2][W];
  const int lane = threadIdx.x % L;
  float w[kHold ? NV * V : 1], b[kHold ? NV * V : 1];
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
#pragma unroll
      for (int j = 0; j < V; ++j) { w[i * V + j] = 1.f; b[i * V + j] = 0.f; }
      if (c < a.d) {
        if (a.w) Vec<RN_F32, V>::load(a.w, c, w + i * V);
        if (a.b) Vec<RN_F32, V>::load(a.b, c, b + i * V);
      }
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
      if (c < a.d) Vec<IN, V>::load(a.x, row * a.xs + c, h + i * V);
    }
    if (a.r) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = V * (lane + L * i);
        if (c < a.d) {
          float t[V];
          Vec<IN, V>::load(a.r, row * a.rs + c, t);
#pragma unroll
          for (int j = 0; j < V; ++j) h[i * V + j] += t[j];
        }
      }
    }
    if (a.sum) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = V * (lane + L * i);
        if (c < a.d) Vec<IN, V>::store(a.sum, row * a.ss + c, h + i * V);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV * V; ++i) s += h[i];
    const float mean = row_sum<W>(s, red[0]) / a.fd;
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[i * V + j] -= mean;
        if (V * (lane + L * i) < a.d) s2 = fmaf(h[i * V + j], h[i * V + j], s2);
      }
    const float rstd = 1.0f / sqrtf(row_sum<W>(s2, red[1]) / a.fd + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (c < a.d) {
        float y[V], wt[V], bt[V];
        if constexpr (!kHold) {
#pragma unroll
          for (int j = 0; j < V; ++j) { wt[j] = 1.f; bt[j] = 0.f; }
          if (a.w) Vec<RN_F32, V>::load(a.w, c, wt);
          if (a.b) Vec<RN_F32, V>::load(a.b, c, bt);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
          y[j] = fmaf(h[i * V + j] * rstd, kHold ? w[i * V + j] : wt[j], kHold ? b[i * V + j] : bt[j]);
        Vec<OUT, V>::store(a.out, row * a.os + c, y);
      }
    }
  }
}

template <int IN, int OUT, int V, int W, int NV>
__global__ void __launch_bounds__(kThreads) norm_rows_backward(NormArgs a) {
  constexpr int L = 64 * W;
  constexpr int R = kThreads / L;
  __shared__ float red[2][2 * W];
  __shared__ float merge[W == 1 ? 64 * NV * V : 1];
  const int lane = threadIdx.x % L;
  float dw[NV * V], db[NV * V];
#pragma unroll
  for (int i = 0; i < NV * V; ++i) { dw[i] = 0.f; db[i] = 0.f; }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / L; row < a.rows; row += step) {
    float x[NV * V], g[NV * V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
#pragma unroll
      for (int j = 0; j < V; ++j) { x[i * V + j] = 0.f; g[i * V + j] = 0.f; }
      if (c < a.d) {
        Vec<IN, V>::load(a.x, row * a.xs + c, x + i * V);
        Vec<OUT, V>::load(a.dout, row * a.os + c, g + i * V);
      }
    }
#pragma unroll
    for (int i = 0; i < NV * V; ++i) s += x[i];
    const float mean = row_sum<W>(s, red[0]) / a.fd;
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[i * V + j] -= mean;
        if (V * (lane + L * i) < a.d) s2 = fmaf(x[i * V + j], x[i * V + j], s2);
      }
    const float rstd = 1.0f / sqrtf(row_sum<W>(s2, red[1]) / a.fd + a.eps);
    float sg = 0.f, sgx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      float wt[V];
#pragma unroll
      for (int j = 0; j < V; ++j) wt[j] = 1.f;
      if (a.w && c < a.d) Vec<RN_F32, V>::load(a.w, c, wt);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = i * V + j;
        x[e] *= rstd;
        if (c < a.d) {
          dw[e] = fmaf(g[e], x[e], dw[e]);
          db[e] += g[e];
          g[e] *= wt[j];
          sg += g[e];
          sgx = fmaf(g[e], x[e], sgx);
        }
      }
    }
    // the first area was last read before the second barrier of this row
    row_sum2<W>(sg, sgx, red[0]);
    sg /= a.fd;
    sgx /= a.fd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (c < a.d) {
        float t[V];
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = 0.f;
        if (a.r) Vec<IN, V>::load(a.r, row * a.rs + c, t);
#pragma unroll
        for (int j = 0; j < V; ++j) t[j] = fmaf(rstd, g[i * V + j] - sg - x[i * V + j] * sgx, t[j]);
        Vec<IN, V>::store(a.sum, row * a.ss + c, t);
      }
    }
    if constexpr (W > 1) __syncthreads();   // the areas are free for the next row
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.d;
  if constexpr (W == 1) {
    // the four waves' sums, added in their order
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float* v = which ? db : dw;
      for (int wv = 0; wv < 4; ++wv) {
        if (static_cast<int>(threadIdx.x >> 6) == wv) {
#pragma unroll
          for (int i = 0; i < NV * V; ++i) {
            float* m = &merge[i * 64 + lane];
            *m = wv == 0 ? v[i] : *m + v[i];
          }
        }
        __syncthreads();
      }
      if (threadIdx.x < 64) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = V * (lane + L * i);
          if (c < a.d) {
#pragma unroll
            for (int j = 0; j < V; ++j) part[static_cast<int64_t>(which) * a.d + c + j] = merge[(i * V + j) * 64 + lane];
          }
        }
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (c < a.d) {
        Vec<RN_F32, V>::store(part, c, dw + i * V);
        Vec<RN_F32, V>::store(part + a.d, c, db + i * V);
      }
    }
  }
}

// dweight and dbias: the partial rows added in the order of their blocks, 16 interleaved
// sums a column which are then added in turn. One block takes 64 columns of the 2 d.
__global__ void __launch_bounds__(1024) norm_reduce(const float* part, int blocks, int d, float* dw, float* db) {
  __shared__ float red[16][64];
  const int col = blockIdx.x * 64 + (threadIdx.x & 63);
  const int grp = threadIdx.x >> 6;
  float s = 0.f;
  if (col < 2 * d)
    for (int i = grp; i < blocks; i += 16) s += part[static_cast<int64_t>(i) * 2 * d + col];
  red[grp][threadIdx.x & 63] = s;
  __syncthreads();
  if (grp == 0 && col < 2 * d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x];
    float* out = col < d ? dw : db;
    if (out) out[col < d ? col : col - d] = s;
  }
}

int backward_blocks(const NormCall& n) {
  // four blocks a CU at most, and at least four rows a block, so that the partial rows
  // (2 d floats a block, written and read once) stay small beside the tensors
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((n.rows + 3) / 4, 512)));
}

template <int IN, int OUT, int V, int W, int NV>
hipError_t launch_one(const NormCall& n, NormArgs a, hipStream_t st) {
  if (!n.backward) {
    constexpr int R = kThreads / (64 * W);
    const int64_t need = (n.rows + R - 1) / R;
    hipLaunchKernelGGL((norm_rows<IN, OUT, V, W, NV>), dim3(static_cast<unsigned>(std::min<int64_t>(need, 2048))),
                       dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  const int blocks = backward_blocks(n);
  hipLaunchKernelGGL((norm_rows_backward<IN, OUT, V, W, NV>), dim3(blocks), dim3(kThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.part) {
    hipLaunchKernelGGL(norm_reduce, dim3((2 * n.d + 63) / 64), dim3(1024), 0, st, a.part, blocks, n.d, n.dw, n.db);
    e = hipGetLastError();
  }
  return e;
}

template <int IN, int OUT>
hipError_t launch_t(const NormCall& n, const NormArgs& a, hipStream_t st) {
  constexpr int V = IN == RN_BF16 ? 8 : 4;   // 16 bytes of the input type
  if (n.vec) {
    const int nv = (n.d / V + 63) / 64;      // vectors a lane of one wave
    if (nv <= 1) return launch_one<IN, OUT, V, 1, 1>(n, a, st);
    if (nv <= 2) return launch_one<IN, OUT, V, 1, 2>(n, a, st);
    if (nv <= 4) return launch_one<IN, OUT, V, 4, 1>(n, a, st);
    if (nv <= 8) return launch_one<IN, OUT, V, 4, 2>(n, a, st);
    if (nv <= 16) return launch_one<IN, OUT, V, 4, 4>(n, a, st);
    if (nv <= 32) return launch_one<IN, OUT, V, 4, 8>(n, a, st);
    if constexpr (V == 4) return launch_one<IN, OUT, V, 4, 16>(n, a, st);
    return hipErrorInvalidValue;
  }
  const int nv = (n.d + 63) / 64;
  if (nv <= 4) return launch_one<IN, OUT, 1, 1, 4>(n, a, st);
  if (nv <= 16) return launch_one<IN, OUT, 1, 4, 4>(n, a, st);
  if (nv <= 32) return launch_one<IN, OUT, 1, 4, 8>(n, a, st);
  if (nv <= 64) return launch_one<IN, OUT, 1, 4, 16>(n, a, st);
  return launch_one<IN, OUT, 1, 4, 64>(n, a, st);
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
