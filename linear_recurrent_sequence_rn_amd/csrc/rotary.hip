// Rotary positions on q and k, one launch for both: pair j of a head's first `rot`
// coordinates is turned by p theta_j and scaled; the coordinates behind are copied.
//
// Bound by HBM (each value read and written once: 16384 tokens of 40 heads of 128, half of each
// turned, bf16: 76 us, 4.4 TB/s; 2 x 2047 tokens of 32 heads of 256 float32: 61 us, 4.4 TB/s) as
// long as the sines stay cheap: an angle
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
constexpr int64_t kGridX = 1 << 23;  // tiles along a grid's x: a launch has fewer than 2^32 threads there

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

// V elements as they are in memory, at any element's address (memory takes them so).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x1 __attribute__((aligned(2)));
template <int DT, int V>
struct Piece {
  static constexpr int kBytes = V * (DT == RN_F32 ? 4 : 2);
  uint32_t u[kBytes < 4 ? 1 : kBytes / 4];
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (kBytes == 16) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p);
      u[0] = x[0]; u[1] = x[1]; u[2] = x[2]; u[3] = x[3];
    } else if constexpr (kBytes == 8) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(p);
      u[0] = x[0]; u[1] = x[1];
    } else if constexpr (kBytes == 4) {
      u[0] = *reinterpret_cast<const u32x1*>(p);
    } else {
      u[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(char* p) const {
    if constexpr (kBytes == 16) *reinterpret_cast<u32x4*>(p) = u32x4{u[0], u[1], u[2], u[3]};
    else if constexpr (kBytes == 8) *reinterpret_cast<u32x2*>(p) = u32x2{u[0], u[1]};
    else if constexpr (kBytes == 4) *reinterpret_cast<u32x1*>(p) = u[0];
    else *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(u[0]);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (DT == RN_F32) f[j] = __uint_as_float(u[j]);
      else f[j] = j % 2 ? __uint_as_float(u[j / 2] & 0xffff0000u) : __uint_as_float(u[j / 2] << 16);
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    if constexpr (DT == RN_F32) {
#pragma unroll
      for (int j = 0; j < V; ++j) u[j] = __float_as_uint(f[j]);
    } else if constexpr (V == 1) {
      u[0] = f32_to_bf16(f[0]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) u[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    }
  }
};

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
  // (what float32 leaves out of the angle, up to 1.2e-7, is made up for to first order: its square
  // is nothing)
  const float x = static_cast<float>(r), rest = static_cast<float>(r - x);
  float s, c;
  sincosf(x, &s, &c);
  return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// `lanes` consecutive threads take one head of one token. A unit of work is two pieces of V
// elements, so placed that neighbouring lanes have neighbouring pieces: with HALF one of each
// half; else, and for the copied rest, one of the first half of the pieces and one of the
// second (where V is 1: the two elements of a pair). Units from `turn` on are copied. The pieces
// of U heads are in flight.
template <int DT, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary(RotArgs a, int lanes) {
  constexpr int U = 4;
  constexpr int E = DT == RN_F32 ? 4 : 2;      // bytes an element
  __shared__ float2 cs[kTable];
  __shared__ int64_t base[kMaxTile][4];   // token offsets: q, k, q_out, k_out
  const int half = a.rot / 2;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x) * a.tile;
  if (row0 >= a.rows) return;
  const int tile = static_cast<int>(min(static_cast<int64_t>(a.tile), a.rows - row0));
  for (int i = threadIdx.x; i < tile * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    const uint32_t row = static_cast<uint32_t>(row0) + t;      // (B * N is below 2^31)
    const uint32_t b = row / static_cast<uint32_t>(a.N), n = row - b * a.N;
    const int64_t p = !a.pos ? a.pos0 + n : a.pos_token ? a.pos[row] : a.pos[b] + n;
    float2 v = angle(p, a.theta[j]);
    v.x *= a.magnitude;
    v.y *= a.inverse ? -a.magnitude : a.magnitude;
    cs[i] = v;
  }
  for (int i = threadIdx.x; i < tile * 4; i += kThreads) {
    const uint32_t row = static_cast<uint32_t>(row0) + i / 4;
    const uint32_t b = row / static_cast<uint32_t>(a.N), n = row - b * a.N;
    base[i / 4][i % 4] = b * a.s[i % 4][0] + n * a.s[i % 4][2];
  }
  __syncthreads();
  const int lane = threadIdx.x & (lanes - 1);
  const int per = kThreads / lanes;
  const int h0 = blockIdx.y * a.heads;
  const int nh = min(a.heads, a.H - h0);
  const int turn = (half + V - 1) / V;           // units of turned elements
  const int copies = (a.d - a.rot + 2 * V - 1) / (2 * V);
  const int units = turn + copies;
  const int second = HALF ? half : V == 1 ? 1 : turn * V;      // from a unit's first piece to its other
  // byte offsets of a unit's pieces in its head, and how many it has
  auto pieces = [&](int u, int* x, int* y) {
    if (u < turn) {
      const int e = V == 1 && !HALF ? 2 * u : u * V;
      *x = e * E;
      *y = (e + second) * E;
      return HALF || e + second < a.rot ? 2 : 1;
    }
    const int e = a.rot + (u - turn) * V;
    *x = e * E;
    *y = (e + copies * V) * E;
    return e + copies * V < a.d ? 2 : 1;
  };
  const int qt = per / nh, qh = per - qt * nh;   // a step of `per` heads in (token, head)
  for (int u = lane; u < units; u += lanes) {
    int ox, oy;
    const int np = pieces(u, &ox, &oy);
    const bool turned = u < turn;
    int i = threadIdx.x / lanes;
    int t = i / nh, h = i - t * nh;
    while (t < tile) {
      Piece<DT, V> x[U], y[U];
      char* out[U];
      int tt[U];
      int n = 0;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (t < tile) {
          const int hd = h0 + h;
          const int isk = hd >= a.Hq;
          const int hh = isk ? hd - a.Hq : hd;
          const char* in = static_cast<const char*>(a.in[isk]) + (base[t][isk] + hh * a.s[isk][1]) * E;
          out[k] = static_cast<char*>(a.out[isk]) + (base[t][2 + isk] + hh * a.s[2 + isk][1]) * E;
          if (!turned && a.in[isk] == a.out[isk]) out[k] = nullptr;   // in place: nothing to copy
          tt[k] = t;
          n = k + 1;
          if (out[k]) x[k].load(in + ox);
          if (out[k] && np == 2) y[k].load(in + oy);
          h += qh;
          t += qt;
          if (h >= nh) { h -= nh; ++t; }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (k < n) {
          if (turned) {
            float p[2 * V];
            x[k].get(p);
            if (np == 2) y[k].get(p + V);
            const float2* c = cs + tt[k] * half;
#pragma unroll
            for (int j = 0; j < V; ++j) {
              // pair j of the unit: one element of each piece, or two of one
              const bool other = !HALF && V > 1 && j >= V / 2;
              if (!other || np == 2) {
                const int e = HALF || V == 1 ? j : 2 * j, f = HALF || V == 1 ? j + V : 2 * j + 1;
                const float2 v = c[HALF || V == 1 ? u * V + j : other ? (u + turn) * (V / 2) + j - V / 2 : u * (V / 2) + j];
                const float re = p[e], im = p[f];
                p[e] = re * v.x - im * v.y;
                p[f] = re * v.y + im * v.x;
              }
            }
            x[k].set(p);
            if (np == 2) y[k].set(p + V);
          }
          if (out[k]) x[k].store(out[k] + ox);
          if (out[k] && np == 2) y[k].store(out[k] + oy);
        }
      }
    }
  }
}

template <int DT>
hipError_t launch_t(const RotaryCall& c, RotArgs& a, hipStream_t st) {
  const int half = a.rot / 2;
  // Elements a piece: the most of 16 bytes that divide every run of coordinates (37 x 222 tokens of
  // 80 heads of 102 bf16, a position per token: 135 us in twos, 244 us one by one).
  int w = DT == RN_BF16 ? 8 : 4;
  while (w > 1 && (a.d % w || (c.half ? half : a.rot) % w)) w /= 2;
  const int units = (half + w - 1) / w + (a.d - a.rot + 2 * w - 1) / (2 * w);
  int lanes = 1;
  while (lanes < units && lanes < 64) lanes *= 2;
  // tokens a block: the angles' cost is shared by all heads whatever the tile, so the tile
  // only has to give every thread work, and 2048 blocks where the call is large enough
  int tile = std::min(kMaxTile, kTable / half);
  while (tile > 1 && (a.rows + tile - 1) / tile < 2048) tile /= 2;
  const int64_t tiles = (a.rows + tile - 1) / tile;
  int groups = 1;
  while (tiles * groups < 512 && groups * 2 * (kThreads / lanes) <= tile * a.H) groups *= 2;
  a.tile = tile;
  a.heads = (a.H + groups - 1) / groups;
  const int64_t x = std::min(tiles, kGridX);
  const dim3 grid(static_cast<unsigned>(x), (a.H + a.heads - 1) / a.heads, static_cast<unsigned>((tiles + x - 1) / x));
#define RN_ROTARY(W)                                                                                             \
  if (w == W) {                                                                                                  \
    if (c.half) hipLaunchKernelGGL((rotary<DT, W, true>), grid, dim3(kThreads), 0, st, a, lanes);                \
    else hipLaunchKernelGGL((rotary<DT, W, false>), grid, dim3(kThreads), 0, st, a, lanes);                      \
  }
  if constexpr (DT == RN_BF16) RN_ROTARY(8)
  RN_ROTARY(4)
  RN_ROTARY(2)
  RN_ROTARY(1)
#undef RN_ROTARY
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
