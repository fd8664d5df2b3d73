// Root-mean-square norm of rows of d values, forward (with the residual sum; an output in float32,
// bf16, or 8 bits with scales) and backward (with the weight's gradient).
//
// Forward, per row: h = x + r; rstd = 1 / sqrt(mean(h^2) + eps); y = h rstd w. In 8 bits, for the whole
// row or each `group` columns of it: scale = max(max|y| / most, 2^-126), out = y / scale rounded to
// nearest even (most: 448 for e4m3, 127 for int8). Backward, with g = dy w: dx = rstd g - x rstd^3
// mean(g x) + dh, dw = sum_rows dy x rstd.
//
// Bound by HBM: every tensor is read or written once (16384 x 4096 bf16 with residual and an e4m3 output with a
// scale for each 128 columns: 90 us, 5.2 TB/s; its gradients 102 us, 5.3 TB/s; a large copy reaches 5.0 to 5.4).
// Smaller calls are bound by latency (32 x 4096, e4m3: kernel 4 us, a call 10; backward of 3001 x 1537 float32 with
// the residual's gradient: a call 22 us, 5 of them the weights' sums). Rows are held as in the layer norm: in the
// registers of 16 lanes, of a wave or of a block, so that the passes over a row (squares, maximum, result) cost no
// memory access; the backward needs one join of a row, for the sums of x x and g x. The largest value of a group of
// 32 to 128 columns is found among the 4 to 32 lanes that hold them, without LDS.
#include <algorithm>

#include "norm_rows.h"
#include "rn_kernels.h"

namespace rn {
namespace {

struct RmsArgs {
  int64_t rows;
  int32_t d, group;           // group: columns a scale; 0 = d
  float eps, fd;              // fd: d
  int64_t xs, rs, ss, os, cs; // row strides: x, residual / dsum, sum_out / dx, out / dout, scale
  const void* x;
  const void* r;              // residual / dsum or null
  const float* w;
  void* sum;                  // sum_out or null / dx
  void* out;
  float* scale;
  const void* dout;
  float* part;                // partial sums of the backward: [blocks][d] or null
};

constexpr bool held8(int dt) { return dt == RN_E4M3 || dt == RN_INT8; }

// The larger of unsigned x over 2^k lanes of a row of 16 (and, with 32, of its neighbour row of 16).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t x, int n) {
  if (n >= 2) x = dpp_max<0xB1>(x);
  if (n >= 4) x = dpp_max<0x4E>(x);
  if (n >= 8) x = dpp_max<0x141>(x);
  if (n >= 16) x = dpp_max<0x140>(x);
  if (n >= 32) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
  if (n >= 64) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 32)));
  return x;
}

// The scale for values of at most |m| (its bits; of a NaN or infinity they are larger than any number's).
template <int OUT>
__device__ __forceinline__ float scale_of(uint32_t m) {
  if (m >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return fmaxf(__uint_as_float(m) / (OUT == RN_E4M3 ? 448.f : 127.f), 1.1754944e-38f);
}

// What a value is divided by its scale with. y (1 / scale) alone is off by up to two roundings, which moves about
// one value in 3e6 that lies beside a border of e4m3 by a step; what it leaves of y, taken exactly, corrects it to
// within 2^-46 before the one rounding. Small scales are raised with their values so that this rest is a
// normal number. (16384 x 4096 bf16, residual, groups of 128, in turn: 95.3 us, as by y (1 / scale);
// by plain divisions 98.5.)
struct Scale {
  float scale, inverse, raise;
  __device__ __forceinline__ explicit Scale(float s) {
    raise = s < 0x1p-90f ? 0x1p64f : 1.f;
    scale = s * raise;
    inverse = 1.f / scale;
  }
  __device__ __forceinline__ float of(float y) const {
    y *= raise;
    const float q = y * inverse;
    return fmaf(fmaf(-q, scale, y), inverse, q);
  }
};

// V consecutive values over their scale in 8 bits (V bytes), at any address; `left` as for Raw.
template <int OUT, int V, Fit FIT>
__device__ __forceinline__ void store8(void* p, int64_t i, int left, const float* y, const Scale& scale) {
  typedef uint32_t u32a __attribute__((aligned(1)));
  uint32_t u[V / 4];
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    if constexpr (OUT == RN_E4M3) {
      u[j] = __builtin_amdgcn_cvt_pk_fp8_f32(scale.of(y[4 * j]), scale.of(y[4 * j + 1]), 0, false);
      u[j] = __builtin_amdgcn_cvt_pk_fp8_f32(scale.of(y[4 * j + 2]), scale.of(y[4 * j + 3]), u[j], true);
    } else {
      u[j] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float t = scale.of(y[4 * j + k]);
        u[j] |= (static_cast<uint32_t>(static_cast<int>(t == t ? rintf(t) : 0.f)) & 0xffu) << (8 * k);
      }
    }
  }
  char* s = static_cast<char*>(p) + i;
  if (FIT == kOdd && left < V) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < left) s[j] = static_cast<char>(u[j / 4] >> (8 * (j % 4)));
  } else {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      if constexpr (FIT == kOdd) reinterpret_cast<u32a*>(s)[j] = u[j];
      else reinterpret_cast<uint32_t*>(s)[j] = u[j];
    }
  }
}

// Thread `lane` of a row's L lanes holds elements [V (lane + L i), +V) for i < NV.
template <int IN, int OUT, int V, int W, int NV, Fit FIT, bool STREAM>
__global__ void __launch_bounds__(threads(W)) rms_rows(RmsArgs a) {
  constexpr int L = lanes(W);
  constexpr int R = threads(W) / L;       // rows per block
  __shared__ float red[2][W ? W : 1];     // rows take the areas in turn
  __shared__ uint32_t top[2][W ? W : 1];
  const int lane = threadIdx.x % L;
  float w[NV * V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = V * (lane + L * i);
#pragma unroll
    for (int j = 0; j < V; ++j) w[i * V + j] = 1.f;
    if ((FIT == kFull || c < a.d) && a.w) load<RN_F32, V, FIT>(a.w, c, a.d - c, w + i * V);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * R + threadIdx.x / L; row < a.rows; row += step, turn ^= 1) {
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
    for (int i = 0; i < NV * V; ++i) s[0] = fmaf(h[i], h[i], s[0]);
    row_sums<W>(s, red[turn]);
    const float rstd = 1.0f / sqrtf(s[0] / a.fd + a.eps);
#pragma unroll
    for (int i = 0; i < NV * V; ++i) h[i] = h[i] * rstd * w[i];
    if constexpr (!held8(OUT)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = V * (lane + L * i);
        if (FIT == kFull || c < a.d) store<OUT, V, FIT, STREAM>(a.out, row * a.os + c, a.d - c, h + i * V);
      }
    } else {
      uint32_t m[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        m[i] = 0;                         // (columns past d are zeros)
#pragma unroll
        for (int j = 0; j < V; ++j) m[i] = max(m[i], __float_as_uint(h[i * V + j]) & 0x7fffffffu);
      }
      if (a.group == 0 || a.group > L * V) {   // one scale a row (a row of at most 128 columns, a group of 128)
#pragma unroll
        for (int i = 1; i < NV; ++i) m[0] = max(m[0], m[i]);
        m[0] = lanes_max(m[0], L > 64 ? 64 : L);
        if constexpr (W > 1) {
          if ((threadIdx.x & 63) == 0) top[turn][threadIdx.x >> 6] = m[0];
          __syncthreads();
#pragma unroll
          for (int i = 0; i < W; ++i) m[0] = max(m[0], top[turn][i]);
        }
        const float sc = scale_of<OUT>(m[0]);
        const Scale by(sc);
        if (lane == 0) a.scale[row * a.cs] = sc;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = V * (lane + L * i);
          if (FIT == kFull || c < a.d) store8<OUT, V, FIT>(a.out, row * a.os + c, a.d - c, h + i * V, by);
        }
      } else {
        const int n = a.group / V;        // lanes a group: a power of two
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = V * (lane + L * i);
          const float sc = scale_of<OUT>(lanes_max(m[i], n));
          const Scale by(sc);
          if (FIT == kFull || c < a.d) {
            if (lane % n == 0) a.scale[row * a.cs + c / a.group] = sc;
            store8<OUT, V, FIT>(a.out, row * a.os + c, a.d - c, h + i * V, by);
          }
        }
      }
    }
  }
}

// The next row's values are on their way while a row is worked on.
template <int IN, int OUT, int V, int W, int NV, Fit FIT, bool STREAM>
__global__ void __launch_bounds__(threads(W)) rms_rows_backward(RmsArgs a) {
  constexpr int L = lanes(W);
  constexpr int R = threads(W) / L;
  constexpr bool kAhead = W < 16 || NV * V <= 4;   // blocks of 16 waves have 128 registers a lane
  __shared__ float red[2][W ? 2 * W : 1];         // rows take the areas in turn
  __shared__ float merge[W <= 1 ? L * NV * V : 1];
  const int lane = threadIdx.x % L;
  float dw[NV * V];
#pragma unroll
  for (int i = 0; i < NV * V; ++i) dw[i] = 0.f;
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
    float m[2] = {0.f, 0.f};              // sums of x x and g w x
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      float wt[V];
#pragma unroll
      for (int j = 0; j < V; ++j) wt[j] = 1.f;
      if ((FIT == kFull || c < a.d) && a.w) load<RN_F32, V, FIT>(a.w, c, a.d - c, wt);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = i * V + j;
        x[e] = rx[i].value(j);
        g[e] = rg[i].value(j);
        t[e] = rr[i].value(j);
        m[0] = fmaf(x[e], x[e], m[0]);
        m[1] = fmaf(g[e] * wt[j], x[e], m[1]);
      }
    }
    if (kAhead && row + step < a.rows) fetch(row + step);
    row_sums<W>(m, red[turn]);
    const float rstd = 1.0f / sqrtf(m[0] / a.fd + a.eps);
    const float sgx = m[1] / a.fd * rstd;       // mean(g xh)
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
          t[e] = fmaf(rstd, g[e] * wt[j] - xh * sgx, t[e]);
        }
        store<IN, V, FIT, STREAM>(a.sum, row * a.ss + c, a.d - c, t + i * V);
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.d;
  if constexpr (W <= 1) {
    // the sums of a wave's rows, then of the four waves, added in their order
    if constexpr (W == 0) {
#pragma unroll
      for (int i = 0; i < NV * V; ++i) { dw[i] += __shfl_xor(dw[i], 16); dw[i] += __shfl_xor(dw[i], 32); }
    }
    for (int wv = 0; wv < 4; ++wv) {
      if (static_cast<int>(threadIdx.x >> 6) == wv && (threadIdx.x & 63) < L) {
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
          float* m = &merge[i * L + lane];
          *m = wv == 0 ? dw[i] : *m + dw[i];
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
            if (FIT != kOdd || c + j < a.d) part[c + j] = merge[(i * V + j) * L + lane];
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = V * (lane + L * i);
      if (FIT == kFull || c < a.d) store<RN_F32, V, FIT>(part, c, a.d - c, dw + i * V);
    }
  }
}

// dweight: the partial rows added in the order of their blocks, 32 interleaved sums a column which
// are then added in turn. One block takes 32 columns.
__global__ void __launch_bounds__(1024) rms_reduce(const float* part, int blocks, int d, float* dw) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  const int grp = threadIdx.x >> 5;
  float s = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int i = grp; i < blocks; i += 32) s += part[static_cast<int64_t>(i) * d + col];
  }
  red[grp][threadIdx.x & 31] = s;
  __syncthreads();
  if (grp == 0 && col < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    dw[col] = s;
  }
}

// Rows that 16 lanes hold in two pieces each: four rows a wave.
bool narrow(const RmsCall& n) { return n.d <= 32 * (n.in_dt == RN_BF16 ? 8 : 4); }

// As the layer norm's: three blocks a CU, and at least four rows a block (16 narrow ones).
int backward_blocks(const RmsCall& n) {
  const int rows = narrow(n) ? 16 : 4;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((n.rows + rows - 1) / rows, 768)));
}

template <int IN, int OUT, int V, int W, int NV, Fit FIT, bool STREAM>
hipError_t launch_full(const RmsCall& n, RmsArgs a, hipStream_t st) {
  if (!n.backward) {
    constexpr int R = threads(W) / lanes(W);
    const int64_t need = (n.rows + R - 1) / R;
    hipLaunchKernelGGL((rms_rows<IN, OUT, V, W, NV, FIT, STREAM>), dim3(static_cast<unsigned>(std::min<int64_t>(need, 2048))),
                       dim3(threads(W)), 0, st, a);
    return hipGetLastError();
  }
  if constexpr (!held8(OUT)) {
    const int blocks = backward_blocks(n);
    hipLaunchKernelGGL((rms_rows_backward<IN, OUT, V, W, NV, FIT, STREAM>), dim3(blocks), dim3(threads(W)), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.part) {
      hipLaunchKernelGGL(rms_reduce, dim3((n.d + 31) / 32), dim3(1024), 0, st, a.part, blocks, n.d, n.dw);
      e = hipGetLastError();
    }
    return e;
  }
  return hipErrorInvalidValue;
}

template <int IN, int OUT, int V, int W, int NV>
hipError_t launch_one(const RmsCall& n, const RmsArgs& a, hipStream_t st) {
  // Past the caches under the layer norm's rule: more bytes than the 256 MB last-level cache, and
  // rows that do not share their 64-byte lines.
  constexpr int in = IN == RN_F32 ? 4 : 2, out = OUT == RN_F32 ? 4 : OUT == RN_BF16 ? 2 : 1;
  const int64_t bytes = n.rows * n.d * (in * (n.r ? 2 : 1) + out + (n.sum ? in : 0));
  const int64_t row = static_cast<int64_t>(n.d) * in;
  const bool stream = bytes > (int64_t(256) << 20) && (row % 64 == 0 || row >= 2048);
  if (!n.vec) return stream ? launch_full<IN, OUT, V, W, NV, kOdd, true>(n, a, st) : launch_full<IN, OUT, V, W, NV, kOdd, false>(n, a, st);
  if (n.d != V * lanes(W) * NV)
    return stream ? launch_full<IN, OUT, V, W, NV, kSome, true>(n, a, st) : launch_full<IN, OUT, V, W, NV, kSome, false>(n, a, st);
  return stream ? launch_full<IN, OUT, V, W, NV, kFull, true>(n, a, st) : launch_full<IN, OUT, V, W, NV, kFull, false>(n, a, st);
}

template <int IN, int OUT>
hipError_t launch_t(const RmsCall& n, const RmsArgs& a, hipStream_t st) {
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

template <int IN>
hipError_t launch_in(const RmsCall& n, const RmsArgs& a, hipStream_t st) {
  switch (n.out_dt) {
    case RN_F32: return launch_t<IN, RN_F32>(n, a, st);
    case RN_BF16: return launch_t<IN, RN_BF16>(n, a, st);
    case RN_E4M3: return launch_t<IN, RN_E4M3>(n, a, st);
    default: return launch_t<IN, RN_INT8>(n, a, st);
  }
}

}  // namespace

size_t rms_backward_ws_bytes(const RmsCall& n) {
  return static_cast<size_t>(backward_blocks(n)) * n.d * sizeof(float);
}

hipError_t launch_rmsnorm(const RmsCall& n, hipStream_t st) {
  RmsArgs a;
  a.rows = n.rows; a.d = n.d; a.group = n.group; a.eps = n.eps; a.fd = static_cast<float>(n.d);
  a.xs = n.xs; a.rs = n.rs; a.ss = n.ss; a.os = n.os; a.cs = n.cs;
  a.x = n.x; a.r = n.r; a.w = n.w; a.sum = n.sum; a.out = n.out; a.scale = n.scale; a.dout = n.dout;
  a.part = n.dw ? static_cast<float*>(n.ws) : nullptr;
  return n.in_dt == RN_F32 ? launch_in<RN_F32>(n, a, st) : launch_in<RN_BF16>(n, a, st);
}

}  // namespace rn
