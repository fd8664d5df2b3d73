// Rotary positions on q and k, one launch for both: pair j of a head's first `rot`
// coordinates is turned by p theta_j and scaled; the coordinates behind are copied.
//
// Bound by HBM (each value read and written once) as long as the sines stay cheap: an angle
// takes a float64 product and reduction and a float32 sine and cosine, about as long as
// moving forty values. So a block takes a few tokens, forms their cosines and sines once,
// in LDS, and turns all heads of these tokens with them. Where that leaves too few
// blocks for the chip, the heads are cut into groups, which form their angles again.
#include <algorithm>

#include "rn_device.h"
#include "rn_kernels.h"

namespace rn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 32;       // tokens a block
constexpr int kTable = 2048;       // cosine/sine pairs in LDS: tile * rot/2 at most

struct RotArgs {
  int32_t N, Hq, H, d, rot;        // H: heads of q and k together
  int32_t tile;                    // tokens a block
  int32_t heads;                   // heads a block
  int64_t rows;                    // B * N
  int64_t pos0;
  const int64_t* pos;
  bool pos_token;
  bool inverse;
  float magnitude;
  int64_t s[4][3];                 // q, k, q_out, k_out: batch, head, token
  const void* in[2];
  void* out[2];
  double theta[kMaxRot / 2];
};

// Reads and writes V elements (16 bytes for V > 1).
template <int DT, int V>
__device__ __forceinline__ void load_v(const void* p, int64_t i, float* f) {
  if constexpr (V == 1) {
    f[0] = Elem<DT>::load(p, i);
  } else if constexpr (DT == RN_F32) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(u[j] << 16);
      f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
}
template <int DT, int V>
__device__ __forceinline__ void store_v(void* p, int64_t i, const float* f) {
  if constexpr (V == 1) {
    Elem<DT>::store(p, i, f[0]);
  } else if constexpr (DT == RN_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

// cos and sin of p theta, both in float64 up to the reduction to [-pi, pi] (as angle_cs,
// with theta in float64: a float32 theta would already be 0.06 rad off at p = 1e6).
__device__ __forceinline__ float2 angle(int64_t p, double theta) {
  const double kTwoPiHi = 6.283185307179586232;
  const double kTwoPiLo = 2.4492935982947064e-16;
  const double kInvTwoPi = 0.15915494309189535;
  const double a = static_cast<double>(p) * theta;
  const double k = rint(a * kInvTwoPi);
  double r = fma(-k, kTwoPiHi, a);
  r = fma(-k, kTwoPiLo, r);
  float2 cs;
  sincosf(static_cast<float>(r), &cs.y, &cs.x);
  return cs;
}

// LANES consecutive threads take one head of one token; V elements an access (pairs of
// scalar accesses where V is 1).
template <int DT, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary(RotArgs a, int lanes) {
  __shared__ float2 cs[kTable];
  const int half = a.rot / 2;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.tile;
  const int tile = static_cast<int>(min(static_cast<int64_t>(a.tile), a.rows - row0));
  for (int i = threadIdx.x; i < tile * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const int64_t row = row0 + t;
    const int64_t b = row / a.N, n = row - b * a.N;
    const int64_t p = !a.pos ? a.pos0 + n : a.pos_token ? a.pos[row] : a.pos[b] + n;
    float2 v = angle(p, a.theta[j]);
    v.x *= a.magnitude;
    v.y *= a.inverse ? -a.magnitude : a.magnitude;
    cs[i] = v;
  }
  __syncthreads();
  const int lane = threadIdx.x & (lanes - 1);
  const int per = kThreads / lanes;
  const int h0 = blockIdx.y * a.heads;
  const int nh = min(a.heads, a.H - h0);
  // units of work of one (token, head): pairs of vectors (or vectors of pairs), then copies
  const int turn = HALF ? half / V : (V == 1 ? half : a.rot / V);
  for (int i = threadIdx.x / lanes; i < tile * nh; i += per) {
    const int t = i / nh, h = h0 + i - t * nh;
    const int64_t row = row0 + t;
    const int64_t b = row / a.N, n = row - b * a.N;
    const int isk = h >= a.Hq;
    const int hh = isk ? h - a.Hq : h;
    const int64_t* si = a.s[isk];
    const int64_t* so = a.s[2 + isk];
    const int64_t x = b * si[0] + hh * si[1] + n * si[2];
    const int64_t y = b * so[0] + hh * so[1] + n * so[2];
    const void* in = a.in[isk];
    void* out = a.out[isk];
    const bool copy = in != out;
    const float2* c = cs + t * half;
    for (int u = lane; u < turn; u += lanes) {
      if constexpr (HALF) {
        float p[V], q[V], f[V], g[V];
        load_v<DT, V>(in, x + u * V, p);
        load_v<DT, V>(in, x + half + u * V, q);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float2 v = c[u * V + j];
          f[j] = p[j] * v.x - q[j] * v.y;
          g[j] = p[j] * v.y + q[j] * v.x;
        }
        store_v<DT, V>(out, y + u * V, f);
        store_v<DT, V>(out, y + half + u * V, g);
      } else if constexpr (V == 1) {
        float p[2], f[2];
        load_v<DT, 1>(in, x + 2 * u, p);
        load_v<DT, 1>(in, x + 2 * u + 1, p + 1);
        const float2 v = c[u];
        f[0] = p[0] * v.x - p[1] * v.y;
        f[1] = p[0] * v.y + p[1] * v.x;
        store_v<DT, 1>(out, y + 2 * u, f);
        store_v<DT, 1>(out, y + 2 * u + 1, f + 1);
      } else {
        float p[V], f[V];
        load_v<DT, V>(in, x + u * V, p);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 v = c[u * (V / 2) + j];
          f[2 * j] = p[2 * j] * v.x - p[2 * j + 1] * v.y;
          f[2 * j + 1] = p[2 * j] * v.y + p[2 * j + 1] * v.x;
        }
        store_v<DT, V>(out, y + u * V, f);
      }
    }
    if (copy)
      for (int e = a.rot + lane * V; e < a.d; e += lanes * V) {
        float p[V];
        load_v<DT, V>(in, x + e, p);
        store_v<DT, V>(out, y + e, p);
      }
  }
}

template <int DT>
hipError_t launch_t(const RotaryCall& c, RotArgs& a, hipStream_t st) {
  constexpr int V = DT == RN_BF16 ? 8 : 4;
  const int half = a.rot / 2;
  // 16-byte accesses need every run of coordinates, stride and pointer in whole vectors
  bool vec = a.d % V == 0 && (c.half ? half % V == 0 : a.rot % V == 0);
  for (int i = 0; i < 2; ++i) {
    if (i == 1 && c.Hk == 0) break;
    vec = vec && reinterpret_cast<uintptr_t>(a.in[i]) % 16 == 0 && reinterpret_cast<uintptr_t>(a.out[i]) % 16 == 0;
    for (int j = 0; j < 3; ++j) vec = vec && a.s[i][j] % V == 0 && a.s[2 + i][j] % V == 0;
  }
  const int w = vec ? V : 1;
  const int units = std::max(c.half ? half / w : std::max(1, a.rot / std::max(w, 2)), (a.d - a.rot + w - 1) / w);
  int lanes = 1;
  while (lanes < units && lanes < 64) lanes *= 2;
  // tokens a block: the angles' cost is shared by all heads whatever the tile, so the tile
  // only has to give every thread work, and 1024 blocks where the call is large enough
  int tile = std::min(kMaxTile, kTable / half);
  while (tile > 1 && (a.rows + tile - 1) / tile < 1024) tile /= 2;
  const int64_t tiles = (a.rows + tile - 1) / tile;
  int groups = 1;
  while (tiles * groups < 512 && groups * 2 * (kThreads / lanes) <= tile * a.H) groups *= 2;
  a.tile = tile;
  a.heads = (a.H + groups - 1) / groups;
  const dim3 grid(static_cast<unsigned>(tiles), (a.H + a.heads - 1) / a.heads);
  if (c.half) {
    if (vec) hipLaunchKernelGGL((rotary<DT, V, true>), grid, dim3(kThreads), 0, st, a, lanes);
    else hipLaunchKernelGGL((rotary<DT, 1, true>), grid, dim3(kThreads), 0, st, a, lanes);
  } else {
    if (vec) hipLaunchKernelGGL((rotary<DT, V, false>), grid, dim3(kThreads), 0, st, a, lanes);
    else hipLaunchKernelGGL((rotary<DT, 1, false>), grid, dim3(kThreads), 0, st, a, lanes);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotaryCall& c, hipStream_t st) {
  RotArgs a;
  a.N = c.N; a.Hq = c.Hq; a.H = c.Hq + c.Hk; a.d = c.d; a.rot = c.rot;
  a.rows = static_cast<int64_t>(c.B) * c.N;
  a.pos0 = c.pos0; a.pos = c.pos; a.pos_token = c.pos_token; a.inverse = c.inverse;
  a.magnitude = c.magnitude;
  for (int j = 0; j < 3; ++j) {
    a.s[0][j] = c.qs[j]; a.s[1][j] = c.ks[j]; a.s[2][j] = c.qos[j]; a.s[3][j] = c.kos[j];
  }
  a.in[0] = c.q; a.in[1] = c.k; a.out[0] = c.q_out; a.out[1] = c.k_out;
  for (int j = 0; j < c.rot / 2; ++j) a.theta[j] = c.theta[j];
  return c.dt == RN_F32 ? launch_t<RN_F32>(c, a, st) : launch_t<RN_BF16>(c, a, st);
}

}  // namespace rn
