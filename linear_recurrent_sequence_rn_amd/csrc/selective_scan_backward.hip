// Gradients of the selective scan (selective_scan.h). With dy = dout z sigmoid(z) (dout without z), and
// g_t the gradient of h_t:
//     g_t = C_t dy_t + a_{t+1} g_{t+1},    a_t = exp(D_t A),    p_t = a_t h_{t-1},   u_t = D_t x_t
//     dC_t = sum_d dy_t h_t,   dB_t = sum_d g_t u_t,   du_t = sum_n g_t B_t
//     dx_t = du_t D_t + skip dy_t,   dD_t = du_t x_t + sum_n g_t p_t A,   ddt_t = dD_t softplus'(dt_t + bias)
//     dA = sum_t g_t p_t D_t,   dskip = sum_t dy_t x_t,   dbias = sum_t ddt_t
//     dz_t = dout y_t (z sigmoid(z))'.
//
// Sequences are cut into pieces. scan_edges gives, for each piece, the state it adds on its own and the
// gradient it passes back on its own; scan_edges_carry joins them along the sequence. Then every piece is taken
// by itself: once forward for the state at each tile's start (kept in LDS), then tile by tile from the last one,
// forward for a tile's decays and states (kept in registers) and back for the gradients. Up to 16 states that
// is scan_piece, whose waves take 64 channels, a lane each, and meet no other; for more, whose starting states
// would not leave LDS for the waves, scan_main, where four waves share the states and join their sums in LDS.
// Lanes are channels, so sums over the wave's 64 channels run across lanes, by a transposing tree: 32 sums of
// 64 lanes, one left in two lanes each, in 71 instructions. Sums over all channels' blocks and over pieces are
// added in a fixed order by scan_sum_tokens and scan_sum_pieces.
//
// Bound by the vector units: 29 instructions a state and token in scan_piece and 10 in scan_edges, of 13 that
// the gradients alone would take (4 x 2048 tokens of 2048 channels x 16 states, bf16 with gate: a call 460 us; under
// the profiler 336 and 90 us, and 55 of joining and sums; busy 69 and 83 %; 250 registers a lane leave two waves a SIMD
// to hide the waits of each other). All of them by four waves a block (scan_main): 640 us for scan_piece's part. Of
// 1024 channels, 16 states 247 us, 32 (scan_main) 632, 64 2086.
#include <algorithm>

#include "selective_scan.h"

namespace rn {
namespace {

struct BackArgs {
  ScanArgs s;                             // its out strides are dout's
  int64_t dxs[2], ddts[2], dzs[2], dbs[3], dcs[3];
  const void* dout;
  const float* dstate_out;                // [S][D][n] or null
  void* dx;
  void* ddt;
  void* dz;
  void* db;
  void* dc;
  float* dA;
  float* dskip;
  float* dbias;
  float* dstate_in;
  float* seg_grad;                        // [pieces][D][n]: the gradient a piece passes back (on its own, then in all)
  float* part_skip;                       // [pieces][D]
  float* part_bias;                       // [pieces][D]
  float* part_bc;                         // [token rows][blocks along channels][2][n]
};

constexpr int kPieceTile = 8, kPieceTiles = 4;   // scan_piece: tokens a tile, tiles a piece at most
// States a wave of scan_main holds: a quarter of them.
int scan_states(int n) { return n <= 32 ? 8 : 16; }
constexpr int tile_of(int NS) { return 32 / NS; }
constexpr int kTiles = 8;                 // scan_main: tiles a piece, at most

// What a block of either kernel works on.
template <int NS>
struct Place {
  Span p;
  int64_t piece;
  int first, nt, last;                    // first token, tokens, the sequence's last piece
  int lane, wave, x, group, d, n0, have, waves;
  bool mine, full;                        // this lane has a channel; every lane has
  __device__ __forceinline__ bool find(const ScanArgs& a) {
    piece = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    x = blockIdx.x;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    group = x / a.tiles;
    const int each = a.D / a.G, in_group = (x - group * a.tiles) * 64 + lane;
    mine = in_group < each;
    full = (x - group * a.tiles) * 64 + 64 <= each;
    d = group * each + in_group;
    n0 = wave * NS;
    have = min(NS, a.n - n0);
    waves = (a.n + NS - 1) / NS;
    if (!seq_place(a.q, piece, &p)) return false;
    p.piece = __builtin_amdgcn_readfirstlane(p.piece);
    const int len = __builtin_amdgcn_readfirstlane(p.len);
    first = p.piece * a.q.len;
    last = len > 0 ? (len - 1) / a.q.len : 0;
    nt = min(len - first, a.q.len);
    return true;
  }
  __device__ __forceinline__ int64_t tokens(const ScanArgs& a, const int64_t* st) const {
    return (a.q.T > 0 ? uniform64(p.row0) * st[1] : p.s * st[0]) + static_cast<int64_t>(first) * st[1] + d;
  }
  __device__ __forceinline__ int64_t groups(const ScanArgs& a, const int64_t* st) const {
    return (a.q.T > 0 ? uniform64(p.row0) * st[2] : p.s * st[0]) + group * st[1] + static_cast<int64_t>(first) * st[2];
  }
  __device__ __forceinline__ int64_t states(const ScanArgs& a, int64_t row) const { return (row * a.D + d) * a.n + n0; }
};

// What a wave works on that holds 64 channels, a lane each (lanes past the group's last channel repeat it).
template <int DT>
struct Lanes {
  typedef typename std::conditional<DT == RN_F32, float, uint16_t>::type elem;
  Span p;
  int64_t piece, row0;
  int first, nt, last, x, group;          // first token, tokens, the sequence's last piece
  unsigned d, c0;                         // channel, the wave's first one
  bool mine, full;                        // this lane has a channel of its own; every lane has
  // A lane's values of a tensor, token after token.
  struct Row {
    const elem* p;
    int64_t step;
    unsigned off;
    __device__ __forceinline__ elem take(unsigned o) {
      const elem v = *reinterpret_cast<const elem*>(reinterpret_cast<const char*>(p) + o);
      p += step;
      return v;
    }
    // N tokens from t0 on; those from `count` (>= 1) on repeat the last one, or are not stored
    template <int N>
    __device__ __forceinline__ void load(int t0, int count, elem (&v)[N]) const {
      const elem* r = p + t0 * step;
      const unsigned o = lane_offset(off);
      if (count >= N) {
#pragma unroll
        for (int t = 0; t < N; ++t, r += step) v[t] = *reinterpret_cast<const elem*>(reinterpret_cast<const char*>(r) + o);
      } else {
#pragma unroll
        for (int t = 0; t < N; ++t) {
          v[t] = *reinterpret_cast<const elem*>(reinterpret_cast<const char*>(r) + o);
          if (t + 1 < count) r += step;
        }
      }
    }
    template <int N>
    __device__ __forceinline__ void store(int t0, int count, const float (&v)[N]) const {
      elem* r = const_cast<elem*>(p + t0 * step);
      const unsigned o = lane_offset(off);
      if (count >= N) {
#pragma unroll
        for (int t = 0; t < N; ++t, r += step) Elem<DT>::store(reinterpret_cast<char*>(r) + o, 0, v[t]);
      } else {
#pragma unroll
        for (int t = 0; t < N; ++t, r += step)
          if (t < count) Elem<DT>::store(reinterpret_cast<char*>(r) + o, 0, v[t]);
      }
    }
    __device__ __forceinline__ void put(int t, float v) const {
      Elem<DT>::store(reinterpret_cast<char*>(const_cast<elem*>(p + t * step)) + off, 0, v);
    }
  };
  __device__ __forceinline__ bool find(const ScanArgs& a, int tile) {
    piece = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    x = tile;
    group = x / a.tiles;
    const int each = a.D / a.G, left = each - (x - group * a.tiles) * 64, lane = threadIdx.x & 63;
    mine = lane < left;
    full = left >= 64;
    c0 = group * each + (each - left);
    d = c0 + min(lane, left - 1);
    if (!seq_place(a.q, piece, &p)) return false;
    p.piece = __builtin_amdgcn_readfirstlane(p.piece);
    row0 = uniform64(p.row0);
    const int len = __builtin_amdgcn_readfirstlane(p.len);
    first = p.piece * a.q.len;
    last = len > 0 ? (len - 1) / a.q.len : 0;
    nt = min(len - first, a.q.len);
    return true;
  }
  __device__ __forceinline__ Row row(bool packed, const void* t, int64_t seq_step, int64_t step) const {
    return Row{static_cast<const elem*>(t) + (packed ? row0 * step : p.s * seq_step) + first * step, step,
               static_cast<unsigned>(d * sizeof(elem))};
  }
  __device__ __forceinline__ Row row(const ScanArgs& a, const void* t, const int64_t* st) const {
    return row(a.q.T > 0, t, st[0], st[1]);
  }
  __device__ __forceinline__ const elem* heads(const ScanArgs& a, const void* t, const int64_t* st) const {
    return static_cast<const elem*>(t) + (a.q.T > 0 ? row0 * st[2] : p.s * st[0]) + group * st[1] + static_cast<int64_t>(first) * st[2];
  }
};

// Values of a token and channel that the scan needs.
struct Inputs {
  float x, dt, z, dout;
};
template <int DT>
__device__ __forceinline__ Inputs fetch_inputs(const BackArgs& a, bool there, int64_t x, int64_t dt, int64_t z, int64_t o) {
  Inputs v = {0.f, 0.f, 0.f, 0.f};
  if (there) {
    v.x = Elem<DT>::load(a.s.x, x);
    v.dt = Elem<DT>::load(a.s.dt, dt);
    if (a.s.z) v.z = Elem<DT>::load(a.s.z, z);
    v.dout = Elem<DT>::load(a.dout, o);
  }
  return v;
}
__device__ __forceinline__ float step_of(const ScanArgs& a, float v) { return a.softplus ? softplus(v) : v; }

// ---- the edges of a piece -------------------------------------------------------------------
// Forward over the piece: the state h it adds, and with P_t = a_1 .. a_t the gradient sum_t P_t C_t dy_t
// that it passes back. A wave takes 64 channels, a lane each, and up to 16 of their states; waves meet
// nowhere.
template <int DT, int NS, bool FAST>
__global__ void __launch_bounds__(256) scan_edges(BackArgs b) {
  constexpr int kGroup = FAST ? 4 : 2;
  const ScanArgs& a = b.s;
  const int sets = (a.n + NS - 1) / NS;
  const int wave = blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Lanes<DT> w;
  if (wave >= a.tiles * a.G * sets || !w.find(a, wave / sets) || w.p.s >= a.q.S || w.last == 0 || w.p.piece > w.last) return;
  const int n0 = (wave % sets) * NS, have = a.n - n0, nt = w.nt;
  float A2[NS], h[NS], P[NS], e[NS];
  load_states<NS>(a.A + static_cast<int64_t>(w.d) * a.n + n0, have, a.a4, A2);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] = in_log2(A2[i]);
    h[i] = e[i] = 0.f;
    P[i] = 1.f;
  }
  const float bias = a.bias ? a.bias[w.d] : 0.f;
  float total = 0.f;
  typename Lanes<DT>::Row x = w.row(a, a.x, a.xs), dt = w.row(a, a.dt, a.dts), dout = w.row(a, b.dout, a.os),
                          z = w.row(a, a.z ? a.z : a.x, a.z ? a.zs : a.xs);
  typename Lanes<DT>::elem nx[kGroup], ndt[kGroup], ndo[kGroup], nz[kGroup] = {};
  auto fetch = [&]() {
    const unsigned o = lane_offset(x.off);
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      nx[k] = x.take(o);
      ndt[k] = dt.take(o);
      ndo[k] = dout.take(o);
    }
    if (a.z) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) nz[k] = z.take(o);
    }
  };
  const typename Lanes<DT>::elem* pb = w.heads(a, a.b, a.bs) + n0;
  const typename Lanes<DT>::elem* pc = w.heads(a, a.c, a.cs) + n0;
  Uniform<DT, NS, FAST> nb, nc;
  nb.load(pb, 0, have);
  nc.load(pc, 0, have);
  auto token = [&](int t, float s, float u, float dy) {
    const Uniform<DT, NS, FAST> B = nb, C = nc;
    if (t + 1 < nt) { pb += a.bs[2]; pc += a.cs[2]; }      // (behind the last token it is read again)
    nb.load(pb, 0, have);
    nc.load(pc, 0, have);
    total += s;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float d = __builtin_amdgcn_exp2f(s * A2[i]);
      h[i] = fmaf(d, h[i], u * B.value(i));
      P[i] *= d;
      e[i] = fmaf(P[i], C.value(i) * dy, e[i]);
    }
  };
  auto gate = [](float v) { return v * sigmoidf(v); };
  const int groups = nt / kGroup;
  if (groups > 0) fetch();
  for (int g = 0; g < groups; ++g) {
    float s[kGroup], u[kGroup], dy[kGroup], zv[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      u[k] = value_of<DT>(nx[k]);
      s[k] = value_of<DT>(ndt[k]) + bias;
      dy[k] = value_of<DT>(ndo[k]);
      zv[k] = value_of<DT>(nz[k]);
    }
    if (g + 1 < groups) fetch();
    if (a.softplus) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) s[k] = softplus(s[k]);
    }
    if (a.z) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) dy[k] *= gate(zv[k]);
    }
#pragma unroll
    for (int k = 0; k < kGroup; ++k) token(g * kGroup + k, s[k], s[k] * u[k], dy[k]);
  }
  for (int t = groups * kGroup; t < nt; ++t) {     // fewer than a group
    const float xv = value_of<DT>(x.take(x.off));
    const float s = step_of(a, value_of<DT>(dt.take(dt.off)) + bias);
    float dy = value_of<DT>(dout.take(dout.off));
    if (a.z) dy *= gate(value_of<DT>(z.take(z.off)));
    token(t, s, s * xv, dy);
  }
  if (!w.mine) return;
  const int64_t to = (w.piece * a.D + w.d) * a.n + n0;
  store_states<NS>(a.seg_state + to, have, a.n % 4 == 0, h);
  store_states<NS>(b.seg_grad + to, have, a.n % 4 == 0, e);
  if (n0 == 0) a.seg_step[w.piece * a.D + w.d] = total;
}

// Along the pieces of sequence blockIdx.y, a thread a state: forward (blockIdx.z = 0), seg_state becomes
// the state a piece starts from; backward, seg_grad the gradient that reaches the token before a piece.
__global__ void __launch_bounds__(256) scan_edges_carry(BackArgs b) {
  const ScanArgs& a = b.s;
  const int s = blockIdx.y;
  Span p;
  seq_span(a.q, s, &p);
  const int pieces = p.len > 0 ? (p.len - 1) / a.q.len + 1 : 1;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, all = static_cast<int64_t>(a.D) * a.n;
  if (pieces < 2 || i >= all) return;
  const int64_t w0 = a.q.T > 0 ? p.row0 / a.q.len + s : static_cast<int64_t>(s) * a.q.n_seg;
  const float A2 = in_log2(a.A[i]);
  const bool back = blockIdx.z;
  const float* first = back ? b.dstate_out : a.state_in;
  float h = first ? first[s * all + i] : 0.f;
  float* to = (back ? b.seg_grad : a.seg_state) + w0 * all + i;
  const float* step = a.seg_step + w0 * a.D + i / a.n;
  constexpr int kAhead = 8;
  for (int g0 = 0; g0 < pieces; g0 += kAhead) {
    float own[kAhead], total[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool there = g0 + k < pieces;
      const int g = back ? pieces - 1 - (g0 + k) : g0 + k;
      own[k] = there ? to[g * all] : 0.f;
      total[k] = there ? step[static_cast<int64_t>(g) * a.D] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int g = back ? pieces - 1 - (g0 + k) : g0 + k;
      const float before = h;
      h = fmaf(__builtin_amdgcn_exp2f(total[k] * A2), h, own[k]);
      if (g0 + k < pieces) to[g * all] = back ? h : before;
    }
  }
}

// ---- a piece --------------------------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
// One level within 16 lanes: lanes whose bit is set keep the second of two values, and each pair of lanes
// exchanges what the other keeps.
template <int CTRL>
__device__ __forceinline__ float fold(float a, float b, bool bit) {
  return (bit ? b : a) + dpp_move<CTRL>(bit ? a : b);
}
// Sums of 64 values over the wave's 64 lanes: lane l receives that of v[l].
__device__ __forceinline__ float sums64(float (&v)[64], int lane) {
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 32]), false, false);
    v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 16]), false, false);
    v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = fold<0x128>(v[k], v[k + 8], lane & 8);      // lane ^ 8
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = fold<0x141>(v[k], v[k + 4], lane & 4);      // lane ^ 7
#pragma unroll
  for (int k = 0; k < 2; ++k) v[k] = fold<0x4E>(v[k], v[k + 2], lane & 2);       // lane ^ 2
  return fold<0xB1>(v[0], v[1], lane & 1);                                       // lane ^ 1
}

// Sums of 32 values over the wave's 64 lanes: lane l receives that of v[l / 2].
__device__ __forceinline__ float sums32(float (&v)[32], int lane) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 16]), false, false);
    v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[k]), __float_as_uint(v[k + 8]), false, false);
    v[k] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = fold<0x128>(v[k], v[k + 4], lane & 8);      // lane ^ 8
#pragma unroll
  for (int k = 0; k < 2; ++k) v[k] = fold<0x141>(v[k], v[k + 2], lane & 4);      // lane ^ 7
  v[0] = fold<0x4E>(v[0], v[1], lane & 2);                                       // lane ^ 2
  return v[0] + dpp_move<0xB1>(v[0]);                                            // lane ^ 1
}

// What a token leaves of a state, a gradient or a sum: nothing where it is behind the sequence's last one, whose
// values it repeats, nor in registers past the n states. (Zeros in their place would not do: what reaches a tile, or
// the token's own values, may be infinite.)
__device__ __forceinline__ float pick(bool there, float now, float before) { return there ? now : before; }
// Nor do lanes past the channels leave anything in sums over the lanes.
template <int N>
__device__ __forceinline__ void leave_out(float (&v)[N], bool mine) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = mine ? v[k] : 0.f;
}

template <int DT, int NS, bool FAST>
__global__ void __launch_bounds__(256, NS <= 8 ? 2 : 1) scan_main(BackArgs b) {
  constexpr int TT = tile_of(NS);
  constexpr int EACH = TT >= 4 ? TT / 4 : 1;
  __shared__ float4 tile[TT][64];                  // D, u, dy
  __shared__ float parts[3][4][TT][64];            // du, the sum of g p A, y: of a wave's states
  __shared__ float starts[kTiles - 1][4][NS][64];  // the state at the start of tiles 1 and on
  const ScanArgs& a = b.s;
  Place<NS> w;
  const bool found = w.find(a);
  if (w.piece >= seq_pieces(a.q)) return;          // (the grid's last row may have more blocks than pieces)
  const int nt = found ? max(w.nt, 0) : 0;
  const int64_t sb = static_cast<int64_t>(w.p.s) * a.D * a.n + static_cast<int64_t>(w.d) * a.n + w.n0;
  const bool real = found && w.p.s < a.q.S;
  float A2[NS], h[NS], e[NS], dA[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) A2[i] = h[i] = e[i] = dA[i] = 0.f;
  float dskip = 0.f, dbias = 0.f;
  const bool ends = real && w.p.piece == w.last;   // the sequence's last piece, if it is empty too
  if (w.mine && real && w.p.piece <= w.last) {
    const float* from = w.p.piece > 0 ? a.seg_state + w.states(a, w.piece) : a.state_in ? a.state_in + sb : nullptr;
    const float* grad = !ends ? b.seg_grad + w.states(a, w.piece + 1) : b.dstate_out ? b.dstate_out + sb : nullptr;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < w.have) {
        A2[i] = in_log2(a.A[static_cast<int64_t>(w.d) * a.n + w.n0 + i]);
        if (from) h[i] = from[i];
        if (grad) e[i] = grad[i];
      }
  }
  if (nt > 0) {
    const float skip = w.mine && a.skip ? a.skip[w.d] : 0.f, bias = w.mine && a.bias ? a.bias[w.d] : 0.f;
    const int64_t xb = w.tokens(a, a.xs), dtb = w.tokens(a, a.dts), zb = w.tokens(a, a.zs), ob = w.tokens(a, a.os);
    const int64_t bb = w.groups(a, a.bs) + w.n0, cb = w.groups(a, a.cs) + w.n0;
    const int64_t dxb = w.tokens(a, b.dxs), ddtb = w.tokens(a, b.ddts), dzb = w.tokens(a, b.dzs);
    const int64_t row = (a.q.T > 0 ? uniform64(w.p.row0) : static_cast<int64_t>(w.p.s) * a.q.N) + w.first;
    const int tiles = (nt + TT - 1) / TT;
    const bool stages = TT >= 4 || w.wave < TT;    // this wave prepares tokens wave * EACH and on of a tile
    Inputs in[EACH];
    auto fetch = [&](int t0) {
#pragma unroll
      for (int k = 0; k < EACH; ++k) {
        const int t = t0 + w.wave * EACH + k;
        in[k] = fetch_inputs<DT>(b, stages && w.mine && t < nt, xb + t * a.xs[1], dtb + t * a.dts[1], zb + t * a.zs[1], ob + t * a.os[1]);
      }
    };
    // ---- forward: the states at the tiles' starts
    fetch(0);
    for (int q = 0; q < tiles - 1; ++q) {
      if (stages) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
          const float s = step_of(a, in[k].dt + bias);
          tile[w.wave * EACH + k][w.lane] = make_float4(s, s * in[k].x, 0.f, 0.f);
        }
      }
      fetch((q + 1) * TT);
      __syncthreads();
      if (w.have > 0) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          Uniform<DT, NS, FAST> B;
          B.load(a.b, bb + (q * TT + t) * a.bs[2], w.have);
          const float4 v = tile[t][w.lane];
#pragma unroll
          for (int i = 0; i < NS; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(v.x * A2[i]), h[i], v.y * B.value(i));
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) starts[q][w.wave][i][w.lane] = h[i];
      }
      __syncthreads();
    }
    // ---- backward, tile by tile
    for (int q = tiles - 1; q >= 0; --q) {
      const int t0 = q * TT;
      float s[EACH], sg[EACH];
      Inputs v[EACH];
#pragma unroll
      for (int k = 0; k < EACH; ++k) {
        const int t = w.wave * EACH + k;
        v[k] = in[k];
        s[k] = step_of(a, in[k].dt + bias);
        sg[k] = a.z ? sigmoidf(in[k].z) : 0.f;
        if (stages) tile[t][w.lane] = make_float4(s[k], s[k] * in[k].x, a.z ? in[k].dout * in[k].z * sg[k] : in[k].dout, 0.f);
      }
      if (q > 0) fetch(t0 - TT);
      __syncthreads();
      if (w.have > 0) {
        if (q > 0) {
#pragma unroll
          for (int i = 0; i < NS; ++i) h[i] = starts[q - 1][w.wave][i][w.lane];
        } else {
#pragma unroll
          for (int i = 0; i < NS; ++i) h[i] = 0.f;
          const float* from = w.p.piece > 0 ? a.seg_state + w.states(a, w.piece) : a.state_in ? a.state_in + sb : nullptr;
          if (w.mine && from) {
#pragma unroll
            for (int i = 0; i < NS; ++i)
              if (i < w.have) h[i] = from[i];
          }
        }
        float sums[64];
        auto tokens = [&](auto whole) {            // whole: every token is one of the sequence's
          constexpr bool kWhole = decltype(whole)::value;
          float dec[TT][NS], p[TT][NS];
          Uniform<DT, NS, FAST> B[TT], C[TT];
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const bool there = kWhole || t0 + t < nt;
            const int at = there ? t0 + t : nt - 1;
            B[t].load(a.b, bb + at * a.bs[2], w.have);
            C[t].load(a.c, cb + at * a.cs[2], w.have);
            const float4 u = tile[t][w.lane];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              const bool has = FAST || i == 0 || i < w.have;
              dec[t][i] = __builtin_amdgcn_exp2f(u.x * A2[i]);
              p[t][i] = dec[t][i] * h[i];
              h[i] = pick(there, fmaf(u.y, B[t].value(i), p[t][i]), h[i]);
              y = pick(has, fmaf(C[t].value(i), h[i], y), y);
              sums[32 + t * NS + i] = u.z * h[i];
            }
            parts[2][w.wave][t][w.lane] = y;
          }
#pragma unroll
          for (int t = TT - 1; t >= 0; --t) {
            const bool there = kWhole || t0 + t < nt;
            const float4 u = tile[t][w.lane];
            float du = 0.f, ws = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              const bool has = FAST || i == 0 || i < w.have;
              const float g = fmaf(C[t].value(i), u.z, e[i]);
              sums[t * NS + i] = g * u.y;
              du = pick(has, fmaf(g, B[t].value(i), du), du);
              const float wp = g * p[t][i];
              ws = pick(has, fmaf(wp, A2[i], ws), ws);
              dA[i] = pick(there, fmaf(wp, u.x, dA[i]), dA[i]);
              e[i] = pick(there, dec[t][i] * g, e[i]);
            }
            parts[0][w.wave][t][w.lane] = du;
            parts[1][w.wave][t][w.lane] = ws;
          }
        };
        if (!FAST || t0 + TT > nt) tokens(std::false_type());
        else tokens(std::true_type());
        if (!w.full) leave_out(sums, w.mine);
        const float total = sums64(sums, w.lane);
        const int r = w.lane & 31, t = r / NS, i = r % NS;
        if (t0 + t < nt && i < w.have)
          b.part_bc[((row + t0 + t) * (static_cast<int64_t>(a.tiles) * a.G) + w.x) * 2 * a.n + (w.lane >> 5) * a.n + w.n0 + i] = total;
      }
      __syncthreads();
      if (stages && w.mine) {
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
          const int t = w.wave * EACH + k;
          if (t0 + t < nt) {
            float du = 0.f, ws = 0.f, y = skip * v[k].x;
            for (int i = 0; i < w.waves; ++i) {
              du += parts[0][i][t][w.lane];
              ws += parts[1][i][t][w.lane];
              y += parts[2][i][t][w.lane];
            }
            float dy = v[k].dout;
            if (a.z) {
              Elem<DT>::store(b.dz, dzb + (t0 + t) * b.dzs[1], dy * y * sg[k] * fmaf(v[k].z, 1.0f - sg[k], 1.0f));
              dy *= v[k].z * sg[k];
            }
            float ddt = fmaf(du, v[k].x, ws * 0.69314718f);
            if (a.softplus) ddt *= sigmoidf(v[k].dt + bias);
            Elem<DT>::store(b.dx, dxb + (t0 + t) * b.dxs[1], fmaf(du, s[k], skip * dy));
            Elem<DT>::store(b.ddt, ddtb + (t0 + t) * b.ddts[1], ddt);
            dskip = fmaf(dy, v[k].x, dskip);
            dbias += ddt;
          }
        }
      }
    }
  }
  if (w.mine) {
    // the piece's own sums (zeros of a piece without tokens), where its starting state was
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < w.have) {
        a.seg_state[w.states(a, w.piece) + i] = dA[i];
        if (real && w.p.piece == 0 && b.dstate_in) b.dstate_in[sb + i] = e[i];
      }
  }
  __syncthreads();
  parts[0][w.wave][0][w.lane] = dskip;
  parts[1][w.wave][0][w.lane] = dbias;
  __syncthreads();
  if (w.wave == 0 && w.mine) {
    dskip = dbias = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dskip += parts[0][i][0][w.lane];
      dbias += parts[1][i][0][w.lane];
    }
    b.part_skip[w.piece * a.D + w.d] = dskip;
    b.part_bias[w.piece * a.D + w.d] = dbias;
  }
  if (a.zero_rest && found && w.mine) {
    const int64_t rows = min(w.p.own - w.first, static_cast<int64_t>(a.q.len));
    const int64_t dxb = w.tokens(a, b.dxs), ddtb = w.tokens(a, b.ddts), dzb = w.tokens(a, b.dzs);
    for (int64_t t = nt + w.wave; t < rows; t += 4) {
      Elem<DT>::store(b.dx, dxb + t * b.dxs[1], 0.f);
      Elem<DT>::store(b.ddt, ddtb + t * b.ddts[1], 0.f);
      if (a.z) Elem<DT>::store(b.dz, dzb + t * b.dzs[1], 0.f);
    }
  }
}

__device__ __forceinline__ void get4(const float4& from, float* v) { v[0] = from.x; v[1] = from.y; v[2] = from.z; v[3] = from.w; }
__device__ __forceinline__ void put4(float4& to, const float* v) { to = make_float4(v[0], v[1], v[2], v[3]); }

// Up to 16 states. A tile's states go four at a time: their decays and states over the tile's 8 tokens are in
// registers, and a lane sums over all of them what its channel needs. What is asked for again at the tile's end
// (its inputs) comes from a cache: held, it would take the registers of the states.
// The kernel's arguments, read again from where the launch put them: what a tile needs of them before and
// behind its states then holds no scalar register in between (held all the time, 250 of them are moved to
// lanes of vector registers and back, 600 of a tile's 3700 instructions).
typedef const __attribute__((address_space(4))) BackArgs* ArgsAgain;
__device__ __forceinline__ ArgsAgain args_again() {
  ArgsAgain p = (ArgsAgain)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

template <int DT, int SETS, bool FAST>
__global__ void __launch_bounds__(64, 2) scan_piece(BackArgs b) {
  constexpr int TT = kPieceTile, NS = 4 * SETS;
  // The state at the start of tiles 1 and on; a tile's is read once, and then replaced by the gradient that
  // reaches the tile before.
  __shared__ float4 starts[kPieceTiles - 1][SETS][64];
  __shared__ float4 own[SETS][64];                       // dA of the piece
  __shared__ float4 decay[SETS][64];                     // A log2(e)
  const ScanArgs& a = b.s;
  Lanes<DT> w;
  const bool found = w.find(a, blockIdx.x);
  if (w.piece >= seq_pieces(a.q)) return;          // (the grid's last row may have more blocks than pieces)
  const int lane = threadIdx.x, n = a.n;
  const bool real = found && w.p.s < a.q.S, fours = n % 4 == 0;
  const int nt = real ? max(w.nt, 0) : 0;
  const int64_t sb = (static_cast<int64_t>(w.p.s) * a.D + w.d) * n, wb = (w.piece * a.D + w.d) * n;
  float dskip = 0.f, dbias = 0.f;
#pragma unroll
  for (int i = 0; i < SETS; ++i) own[i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* from = nullptr;                     // the starting state
  const float* grad = nullptr;                     // and the gradient that reaches the piece from behind
  if (real && w.p.piece <= w.last) {
    const bool ends = w.p.piece == w.last;         // the sequence's last piece, if it is empty too
    grad = !ends ? b.seg_grad + wb + static_cast<int64_t>(a.D) * n : b.dstate_out ? b.dstate_out + sb : nullptr;
    from = w.p.piece > 0 ? a.seg_state + wb : a.state_in ? a.state_in + sb : nullptr;
  }
  float* const passed = real && w.p.piece == 0 && w.mine && b.dstate_in ? b.dstate_in + sb : nullptr;
  if (passed && nt == 0) {                         // a sequence without tokens
    float e[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) e[i] = 0.f;
    if (grad) load_states<NS>(grad, n, fours, e);
    store_states<NS>(passed, n, fours, e);
  }
  if (nt > 0) {
    const float skip = a.skip ? a.skip[w.d] : 0.f, bias = a.bias ? a.bias[w.d] : 0.f;
    typedef typename Lanes<DT>::elem elem;
    const elem* pb = w.heads(a, a.b, a.bs);
    const elem* pc = w.heads(a, a.c, a.cs);
    const auto x = w.row(a, a.x, a.xs), dt = w.row(a, a.dt, a.dts), dout = w.row(a, b.dout, a.os),
               z = w.row(a, a.z ? a.z : a.x, a.z ? a.zs : a.xs);
    // every row of the piece is asked for at once, a lane a row, so that the loads below find it in a cache
    elem asked[2];
    {
      const int64_t t = min(lane & 31, nt - 1);
      const unsigned half = lane >> 5;
      asked[0] = half ? x.p[t * x.step + w.c0] : dt.p[t * dt.step + w.c0];
      asked[1] = half ? dout.p[t * dout.step + w.c0] : z.p[t * z.step + w.c0];
    }
    const int tiles = (nt + TT - 1) / TT;
    const float* const A = a.A + static_cast<int64_t>(w.d) * n;
    float A2[NS];
    load_states<NS>(A, n, a.a4, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] = in_log2(A2[i]);
#pragma unroll
    for (int i = 0; i < SETS; ++i) put4(decay[i][lane], A2 + 4 * i);
    // ---- forward: the states at the tiles' starts
    if (tiles > 1) {
      float h[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) h[i] = 0.f;
      if (from) load_states<NS>(from, n, fours, h);
      elem nx[TT], ndt[TT];
      x.load(0, TT, nx);
      dt.load(0, TT, ndt);
      for (int q = 0; q < tiles - 1; ++q) {
        float s[TT], u[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          u[t] = value_of<DT>(nx[t]);
          s[t] = value_of<DT>(ndt[t]) + bias;
        }
        if (q + 2 < tiles) {
          x.load((q + 1) * TT, TT, nx);
          dt.load((q + 1) * TT, TT, ndt);
        }
        if (a.softplus) {
#pragma unroll
          for (int t = 0; t < TT; ++t) s[t] = softplus(s[t]);
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) u[t] *= s[t];
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          Uniform<DT, NS, FAST> B;
          B.load(pb, (q * TT + t) * a.bs[2], n);
#pragma unroll
          for (int i = 0; i < NS; ++i) h[i] = fmaf(__builtin_amdgcn_exp2f(s[t] * A2[i]), h[i], u[t] * B.value(i));
        }
#pragma unroll
        for (int i = 0; i < SETS; ++i) put4(starts[q][i][lane], h + 4 * i);
      }
    }
    asm volatile("" ::"v"(asked[0]), "v"(asked[1]));
    // ---- backward, tile by tile
    const int64_t bc_step = static_cast<int64_t>(a.tiles) * a.G * 2 * n;
    float* bc = b.part_bc + ((a.q.T > 0 ? w.row0 : static_cast<int64_t>(w.p.s) * a.q.N) + w.first) * bc_step +
                w.x * 2 * n + (lane & 1) * n;
    struct Raw { elem x[TT], dt[TT], dout[TT], z[TT]; };
    auto inputs = [&](ArgsAgain k, int t0, int count, Raw& r) {
      const bool packed = k->s.q.T > 0, gate = k->s.z;
      w.row(packed, k->s.x, k->s.xs[0], k->s.xs[1]).load(t0, count, r.x);
      w.row(packed, k->s.dt, k->s.dts[0], k->s.dts[1]).load(t0, count, r.dt);
      w.row(packed, k->dout, k->s.os[0], k->s.os[1]).load(t0, count, r.dout);
      w.row(packed, gate ? k->s.z : k->s.x, gate ? k->s.zs[0] : k->s.xs[0], gate ? k->s.zs[1] : k->s.xs[1]).load(t0, count, r.z);
    };
    Raw next;
    inputs(args_again(), (tiles - 1) * TT, nt - (tiles - 1) * TT, next);
    for (int q = tiles - 1; q >= 0; --q) {
      const int t0 = q * TT, count = min(nt - t0, TT);
      float s[TT], u[TT], dy[TT], du[TT], ws[TT], y[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        u[t] = value_of<DT>(next.x[t]);
        s[t] = value_of<DT>(next.dt[t]) + bias;
        dy[t] = value_of<DT>(next.dout[t]);
        y[t] = value_of<DT>(next.z[t]);
      }
      if (a.z) {
#pragma unroll
        for (int t = 0; t < TT; ++t) dy[t] *= y[t] * sigmoidf(y[t]);
      }
      if (a.softplus) {
#pragma unroll
        for (int t = 0; t < TT; ++t) s[t] = softplus(s[t]);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        du[t] = ws[t] = y[t] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) u[t] *= s[t];
      // whole: every token is one of the sequence's. (Where the lanes load B and C for themselves the other form
      // serves both: two forms' registers spill more, 5 states, 4 x 2048 tokens of 1024 channels 481 us and 442.)
      auto states = [&](auto whole) {
        constexpr bool kWhole = decltype(whole)::value;
#pragma unroll 1
        for (int c = 0; c < NS; c += 4) {
          float A2[4], h[4], e[4], dec[TT][4], p[TT][4], sums[32];
          Uniform<DT, 4, FAST> B[TT], C[TT];
          {
            const elem* rb = pb + t0 * a.bs[2] + c;
            const elem* rc = pc + t0 * a.cs[2] + c;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
              B[t].load(rb, 0, n - c);
              C[t].load(rc, 0, n - c);
              rb += t + 1 < count ? a.bs[2] : 0;
              rc += t + 1 < count ? a.cs[2] : 0;
            }
          }
          get4(decay[c / 4][lane], A2);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = e[i] = 0.f;
          if (q == tiles - 1) {
            if (grad) load_states<4>(grad + c, n - c, fours, e);
          } else {
            get4(starts[q][c / 4][lane], e);
          }
          if (q == 0) {
            if (from) load_states<4>(from + c, n - c, fours, h);
          } else {
            get4(starts[q - 1][c / 4][lane], h);
          }
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const bool there = kWhole || t < count;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool has = FAST || i == 0 || c + i < n;
              dec[t][i] = __builtin_amdgcn_exp2f(s[t] * A2[i]);
              p[t][i] = dec[t][i] * h[i];
              h[i] = pick(there, fmaf(u[t], B[t].value(i), p[t][i]), h[i]);
              y[t] = pick(has, fmaf(C[t].value(i), h[i], y[t]), y[t]);
              sums[t * 4 + i] = dy[t] * h[i];
            }
          }
          if (!w.full) leave_out(sums, w.mine);
          const float sum_c = sums32(sums, lane);
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            B[t].fresh();
            C[t].fresh();
          }
          float dA[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int t = TT - 1; t >= 0; --t) {
            const bool there = kWhole || t < count;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool has = FAST || i == 0 || c + i < n;
              const float g = fmaf(C[t].value(i), dy[t], e[i]);
              sums[t * 4 + i] = g * u[t];
              du[t] = pick(has, fmaf(g, B[t].value(i), du[t]), du[t]);
              const float wp = g * p[t][i];
              ws[t] = pick(has, fmaf(wp, A2[i], ws[t]), ws[t]);
              dA[i] = pick(there, fmaf(wp, s[t], dA[i]), dA[i]);
              e[i] = pick(there, dec[t][i] * g, e[i]);
            }
          }
          float sum[4];
          get4(own[c / 4][lane], sum);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] += dA[i];
          put4(own[c / 4][lane], sum);
          if (q > 0) put4(starts[q - 1][c / 4][lane], e);
          if (q == 0 && passed) store_states<4>(passed + c, n - c, fours, e);
          if (!w.full) leave_out(sums, w.mine);
          const float sum_b = sums32(sums, lane);
          const int t = lane >> 3, i = c + (lane >> 1 & 3);
          if (t < count && i < n) bc[(t0 + t) * bc_step + i] = lane & 1 ? sum_c : sum_b;
        }
      };
      if (!FAST || count < TT) states(std::false_type());
      else states(std::true_type());
      // what belongs to a channel and token, while the next tile's inputs are on their way
      Raw r;
      const ArgsAgain k = args_again();
      const bool packed = k->s.q.T > 0;
      inputs(k, t0, count, r);
      if (q > 0) inputs(k, t0 - TT, TT, next);
      if (count < TT) {                            // (no 0 x of a token behind the last one: x may be infinite)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t >= count) {
            s[t] = dy[t] = du[t] = ws[t] = 0.f;
            r.x[t] = 0;
          }
      }
      float g[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float xv = value_of<DT>(r.x[t]), slope = a.softplus ? sigmoidf(value_of<DT>(r.dt[t]) + bias) : 1.f;
        g[t] = fmaf(du[t], xv, ws[t] * 0.69314718f) * slope;
        du[t] = fmaf(du[t], s[t], skip * dy[t]);
        dskip = fmaf(dy[t], xv, dskip);
        dbias += g[t];
        y[t] = fmaf(skip, xv, y[t]);
      }
      if (w.mine) {
        w.row(packed, k->dx, k->dxs[0], k->dxs[1]).store(t0, count, du);
        w.row(packed, k->ddt, k->ddts[0], k->ddts[1]).store(t0, count, g);
      }
      if (k->s.z) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const float zv = value_of<DT>(r.z[t]), sg = sigmoidf(zv);
          y[t] *= value_of<DT>(r.dout[t]) * sg * fmaf(zv, 1.0f - sg, 1.0f);
        }
        if (w.mine) w.row(packed, k->dz, k->dzs[0], k->dzs[1]).store(t0, count, y);
      }
    }
  }
  if (!w.mine) return;
  // the piece's own sums (zeros of a piece without tokens), where its starting state was
  float dA[NS];
#pragma unroll
  for (int i = 0; i < SETS; ++i) get4(own[i][lane], dA + 4 * i);
  store_states<NS>(a.seg_state + wb, n, fours, dA);
  b.part_skip[w.piece * a.D + w.d] = dskip;
  b.part_bias[w.piece * a.D + w.d] = dbias;
  if (a.zero_rest && found) {
    const auto dx = w.row(a, b.dx, b.dxs), ddt = w.row(a, b.ddt, b.ddts), dz = w.row(a, a.z ? b.dz : b.dx, a.z ? b.dzs : b.dxs);
    const int rows = static_cast<int>(min(w.p.own - w.first, static_cast<int64_t>(a.q.len)));
    for (int t = nt; t < rows; ++t) {
      dx.put(t, 0.f);
      ddt.put(t, 0.f);
      if (a.z) dz.put(t, 0.f);
    }
  }
}

// ---- sums over blocks -----------------------------------------------------------------------

// dB and dC of a piece's tokens: the blocks along the channels of a group, in their order.
template <int DT>
__global__ void __launch_bounds__(256) scan_sum_tokens(BackArgs b) {
  const ScanArgs& a = b.s;
  Span p;
  if (!seq_place(a.q, blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y, &p)) return;
  const int64_t first = static_cast<int64_t>(p.piece) * a.q.len;
  const int64_t rows = min(p.own - first, static_cast<int64_t>(a.q.len));
  const int per = 2 * a.n * a.G;
  const int64_t row = (a.q.T > 0 ? p.row0 : static_cast<int64_t>(p.s) * a.q.N) + first;
  const int64_t bb = (a.q.T > 0 ? p.row0 * b.dbs[2] : p.s * b.dbs[0]) + first * b.dbs[2];
  const int64_t cb = (a.q.T > 0 ? p.row0 * b.dcs[2] : p.s * b.dcs[0]) + first * b.dcs[2];
  for (int64_t i = threadIdx.x; i < rows * per; i += 256) {
    const int64_t t = i / per;
    const int k = static_cast<int>(i - t * per), g = k / (2 * a.n), c = k - g * 2 * a.n;
    float s = 0.f;
    if (first + t < p.len) {
      const float* from = b.part_bc + ((row + t) * a.G + g) * a.tiles * 2 * a.n + c;
#pragma unroll 4
      for (int x = 0; x < a.tiles; ++x) s += from[static_cast<int64_t>(x) * 2 * a.n];
    } else if (!a.zero_rest) {
      continue;
    }
    if (c < a.n) Elem<DT>::store(b.db, bb + t * b.dbs[2] + g * b.dbs[1] + c, s);
    else Elem<DT>::store(b.dc, cb + t * b.dcs[2] + g * b.dcs[1] + c - a.n, s);
  }
}

// dA, dskip and dbias: the pieces' sums in 32 interleaved ones a column, which are then added in turn.
__global__ void __launch_bounds__(1024) scan_sum_pieces(BackArgs b, int64_t pieces) {
  __shared__ float red[32][33];
  const ScanArgs& a = b.s;
  const int64_t all = static_cast<int64_t>(a.D) * a.n;
  int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const float* from = nullptr;
  float* to = nullptr;
  int64_t step = a.D;
  if (col < all) { from = a.seg_state; to = b.dA; step = all; }
  else if ((col -= all) < a.D) { from = b.part_skip; to = b.dskip; }
  else if ((col -= a.D) < a.D) { from = b.part_bias; to = b.dbias; }
  const int grp = threadIdx.x >> 5;
  float s = 0.f;
  if (to) {
#pragma unroll 4
    for (int64_t i = grp; i < pieces; i += 32) s += from[i * step + col];
  }
  red[grp][threadIdx.x & 31] = s;
  __syncthreads();
  if (grp == 0 && to) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    to[col] = s;
  }
}

template <int DT, int NS>
hipError_t launch_edges(const BackArgs& b, hipStream_t st) {
  const ScanArgs& a = b.s;
  const int64_t x = static_cast<int64_t>(a.tiles) * a.G * ((a.n + NS - 1) / NS);
  const int waves = static_cast<int>(std::min<int64_t>(x, 4));
  const dim3 grid = seq_grid(a.q, (x + waves - 1) / waves), block(64 * waves);
  if (scan_fast(a, DT, NS)) hipLaunchKernelGGL((scan_edges<DT, NS, true>), grid, block, 0, st, b);
  else hipLaunchKernelGGL((scan_edges<DT, NS, false>), grid, block, 0, st, b);
  return hipGetLastError();
}
template <int DT, int SETS>
hipError_t launch_piece(const BackArgs& b, hipStream_t st) {
  const dim3 grid = seq_grid(b.s.q, static_cast<int64_t>(b.s.tiles) * b.s.G);
  if (scan_fast(b.s, DT, 4 * SETS)) hipLaunchKernelGGL((scan_piece<DT, SETS, true>), grid, dim3(64), 0, st, b);
  else hipLaunchKernelGGL((scan_piece<DT, SETS, false>), grid, dim3(64), 0, st, b);
  return hipGetLastError();
}
template <int DT, int NS>
hipError_t launch_main(const BackArgs& b, hipStream_t st) {
  const dim3 grid = seq_grid(b.s.q, static_cast<int64_t>(b.s.tiles) * b.s.G);
  if (scan_fast(b.s, DT, NS)) hipLaunchKernelGGL((scan_main<DT, NS, true>), grid, dim3(256), 0, st, b);
  else hipLaunchKernelGGL((scan_main<DT, NS, false>), grid, dim3(256), 0, st, b);
  return hipGetLastError();
}
template <int DT>
hipError_t launch_back(const BackArgs& b, hipStream_t st) {
  const ScanArgs& a = b.s;
  const int64_t all = static_cast<int64_t>(a.D) * a.n;
  hipError_t e;
  if (a.q.N > a.q.len) {
    e = a.n <= 4 ? launch_edges<DT, 4>(b, st) : a.n <= 8 ? launch_edges<DT, 8>(b, st) : a.n % 12 == 0 ? launch_edges<DT, 12>(b, st)
                                                                                      : launch_edges<DT, 16>(b, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_edges_carry, dim3(static_cast<unsigned>((all + 255) / 256), a.q.S, 2), dim3(256), 0, st, b);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  e = a.n <= 4    ? launch_piece<DT, 1>(b, st)
      : a.n <= 8  ? launch_piece<DT, 2>(b, st)
      : a.n <= 12 ? launch_piece<DT, 3>(b, st)
      : a.n <= 16 ? launch_piece<DT, 4>(b, st)
      : a.n <= 32 ? launch_main<DT, 8>(b, st)
                  : launch_main<DT, 16>(b, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((scan_sum_tokens<DT>), seq_grid(a.q, 1), dim3(256), 0, st, b);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(scan_sum_pieces, dim3(static_cast<unsigned>((all + 2 * a.D + 31) / 32)), dim3(1024), 0, st, b, seq_pieces(a.q));
  return hipGetLastError();
}

// Floats of each part of the workspace.
struct Parts {
  size_t state, step, bc;
  explicit Parts(const ScanArgs& a) {
    const size_t rows = static_cast<size_t>(seq_pieces(a.q));
    const size_t tokens = a.q.T > 0 ? static_cast<size_t>(a.q.T) : static_cast<size_t>(a.q.S) * a.q.N;
    state = rows * a.D * a.n;
    step = rows * a.D;
    bc = tokens * a.tiles * a.G * 2 * a.n;
  }
  size_t all() const { return 2 * state + 3 * step + bc; }
};
// Tokens a piece: the most that leave waves for the chip to hold at once, two a SIMD (float32, 5 sequences of
// 1501 tokens in all, 212 channels: 8 tokens 59 us, 32 110; bf16, 16 states, 4 x 512 tokens of 1024 channels: 8
// tokens 102, 16 95, 32 135; 4 x 2048 of 2048: 663, 532 and 484, which whole tiles in a form of their own made 460).
// scan_main's blocks are four waves.
ScanArgs pieces_of(const ScanCall& c) {
  const bool small = c.n <= 16;
  const int tile = small ? kPieceTile : tile_of(scan_states(c.n));
  const int64_t per = static_cast<int64_t>(c.G) * ((c.D / c.G + 63) / 64);
  const int64_t tokens = c.T > 0 ? c.T : static_cast<int64_t>(c.S) * c.N;
  int len = tile * (small ? kPieceTiles : kTiles);
  while (len > tile && tokens * per < (small ? 2048 : 512) * static_cast<int64_t>(len)) len /= 2;
  return scan_args(c, len);
}

}  // namespace

size_t scan_backward_ws_bytes(const ScanCall& c) { return Parts(pieces_of(c)).all() * sizeof(float); }

hipError_t launch_selective_backward(const ScanCall& c, const ScanGrads& g, hipStream_t st) {
  BackArgs b;
  b.s = pieces_of(c);
  for (int i = 0; i < 2; ++i) { b.dxs[i] = g.dxs[i]; b.ddts[i] = g.ddts[i]; b.dzs[i] = g.dzs[i]; }
  for (int i = 0; i < 3; ++i) { b.dbs[i] = g.dbs[i]; b.dcs[i] = g.dcs[i]; }
  b.dout = g.dout; b.dstate_out = g.dstate_out; b.dx = g.dx; b.ddt = g.ddt; b.dz = g.dz; b.db = g.db; b.dc = g.dc;
  b.dA = g.dA; b.dskip = g.dskip; b.dbias = g.dbias; b.dstate_in = g.dstate_in;
  const Parts parts(b.s);
  float* ws = static_cast<float*>(c.ws);
  b.s.seg_state = ws;
  b.seg_grad = ws + parts.state;
  b.s.seg_step = b.seg_grad + parts.state;
  b.part_skip = b.s.seg_step + parts.step;
  b.part_bias = b.part_skip + parts.step;
  b.part_bc = b.part_bias + parts.step;
  return c.type == RN_F32 ? launch_back<RN_F32>(b, st) : launch_back<RN_BF16>(b, st);
}

}  // namespace rn
