// Selective scan: prompts (selective_scan.h) and single tokens.
//
// Prompts. Bound by the vector units: a state takes 5 instructions a token (the exponent, its exponential, which
// counts twice, the input's product, and the two sums; 4 where only states are wanted), a channel 37 more (counted:
// softplus 16, gate 8, loads, the skip and the output 13; 25 where only states are wanted). A wave has 64 channels
// with all their states in its lanes' registers, B and C in its scalar ones, and nothing to share with other waves: no
// LDS, no barrier (sharing a channel's states over four waves, joined in LDS, took 547 us where this takes 228). A
// sequence whose channels do not fill the chip is cut into segments: one pass gives the state that each adds on its
// own, scan_carry carries the states over the segments, a second pass gives the outputs (8192 tokens of 4096 channels
// x 16 states, bf16 with gate: 106, 17 and 138 us under the profiler; vector units 91 and 93 % busy). 32 sequences of
// 512 tokens need no cut: 295 us for twice the tokens. 32 states of 2048 channels take 241 us, 64 take 617: B and C of
// more than 16 states are waited for, a set at a time.
//
// Single tokens. Bound by HBM: the float32 state is read and written once.
#include <algorithm>

#include "norm_rows.h"
#include "selective_scan.h"

namespace rn {
namespace {

// Where a kernel starts and ends: a whole sequence, or a segment whose starting state is in the
// workspace; or the state a segment adds on its own.
enum ScanMode : int { kScanOut = 0, kScanState = 1 };

// A wave takes 64 channels of a group, a lane each with all its states, and a piece of a sequence. Waves
// meet nowhere. Tokens go in groups, the next group's values on their way.
template <int DT, int NS, bool FAST, ScanMode MODE>
__global__ void __launch_bounds__(256) scan_rows(ScanArgs a) {
  constexpr int CH = !FAST ? 4 : NS <= 16 ? NS : NS % 16 ? 12 : 16;   // states whose B and C are held at once
  constexpr int kGroup = NS > 16 || !FAST ? 2 : 4;
  typedef typename std::conditional<DT == RN_F32, float, uint16_t>::type elem;
  Span p;
  const int64_t piece = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
  const int x = blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (x >= a.tiles * a.G || !seq_place(a.q, piece, &p)) return;
  p.piece = __builtin_amdgcn_readfirstlane(p.piece);
  const int len = __builtin_amdgcn_readfirstlane(p.len);
  const int first = p.piece * a.q.len;
  const int last = len > 0 ? (len - 1) / a.q.len : 0;      // the piece that ends the sequence
  if (MODE == kScanState && p.piece >= last) return;
  const int nt = min(len - first, a.q.len);                // tokens of the piece
  const int group = x / a.tiles, each = a.D / a.G, left = each - (x - group * a.tiles) * 64;
  const int lane = threadIdx.x & 63;
  const bool mine = lane < left;
  const unsigned d = group * each + (each - left) + min(lane, left - 1);     // (lanes past the last channel repeat it)
  const unsigned off = d * sizeof(elem);
  const int64_t row0 = uniform64(p.row0);
  auto at = [&](const void* t, const int64_t* st) {        // the piece's first row
    return static_cast<const elem*>(t) + ((a.q.T > 0 ? row0 : static_cast<int64_t>(first)) * st[1] +
                                          (a.q.T > 0 ? first * st[1] : p.s * st[0]));
  };
  auto heads = [&](const int64_t* st) {
    return (a.q.T > 0 ? row0 * st[2] : p.s * st[0]) + group * st[1] + static_cast<int64_t>(first) * st[2];
  };
  const elem* px = at(a.x, a.xs);
  const elem* pdt = at(a.dt, a.dts);
  const elem* pz = MODE == kScanOut && a.z ? at(a.z, a.zs) : nullptr;
  const elem* pb = static_cast<const elem*>(a.b) + heads(a.bs);
  const elem* pc = static_cast<const elem*>(a.c) + heads(a.cs);
  float A2[NS], h[NS];
  load_states<NS>(a.A + static_cast<int64_t>(d) * a.n, a.n, a.a4, A2);
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] = in_log2(A2[i]);
    h[i] = 0.f;
  }
  const float skip = a.skip ? a.skip[d] : 0.f, bias = a.bias ? a.bias[d] : 0.f;
  const int slot = p.s < a.q.S ? seq_slot(a.slots, a.n_slots, p.s) : -1;
  const int64_t sb = (static_cast<int64_t>(slot) * a.D + d) * a.n;
  if (MODE == kScanOut) {
    const float* from = p.piece <= last && last > 0 ? a.seg_state + (piece * a.D + d) * a.n
                        : slot >= 0 && a.state_in && p.piece == 0 ? a.state_in + sb : nullptr;
    if (from) load_states<NS>(from, a.n, a.n % 4 == 0, h);
  }
  elem* out = MODE == kScanOut ? const_cast<elem*>(at(a.out, a.os)) : nullptr;
  float total = 0.f;                      // kScanState: the sum of D_t
  elem nx[kGroup], ndt[kGroup], nz[kGroup] = {};
  auto take = [](const elem*& p, int64_t step, unsigned o) {   // the lane's value of the row p stands at
    const elem v = *reinterpret_cast<const elem*>(reinterpret_cast<const char*>(p) + o);
    p += step;
    return v;
  };
  auto fetch = [&]() {                    // the next group's values
    const unsigned o = lane_offset(off);
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      nx[k] = take(px, a.xs[1], o);
      ndt[k] = take(pdt, a.dts[1], o);
    }
    if (MODE == kScanOut && pz) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) nz[k] = take(pz, a.zs[1], o);
    }
  };
  // Up to 16 states' B and C are on their way while the token before is worked on; of more, each set's when
  // it is needed.
  constexpr bool kAhead = NS == CH && FAST;
  Uniform<DT, CH, FAST> nb, nc;
  auto heads_of = [&](int c, Uniform<DT, CH, FAST>* B, Uniform<DT, CH, FAST>* C) {
    B->load(pb, c, a.n - c);
    if (MODE == kScanOut) C->load(pc, c, a.n - c);
  };
  auto token = [&](float xv, float s, int t) {
    const float u = s * xv;
    float y = skip * xv;
    Uniform<DT, CH, FAST> B, C;
    if (kAhead) {
      B = nb;
      C = nc;
      if (t + 1 < nt) { pb += a.bs[2]; pc += a.cs[2]; }      // (behind the last token it is read again)
      heads_of(0, &nb, &nc);
    }
#pragma unroll
    for (int c = 0; c < NS; c += CH) {
      if (!kAhead) heads_of(c, &B, &C);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        h[c + i] = fmaf(__builtin_amdgcn_exp2f(s * A2[c + i]), h[c + i], u * B.value(i));
        // (registers past the n states hold 0 times the token's values: NaN where those are infinite)
        if (MODE == kScanOut) y = fmaf(C.value(i), FAST || c + i < a.n ? h[c + i] : 0.f, y);
      }
    }
    if (!kAhead) { pb += a.bs[2]; pc += a.cs[2]; }
    if (MODE == kScanState) total += s;
    return y;
  };
  const int groups = nt > 0 ? nt / kGroup : 0;
  if (groups > 0) fetch();
  if (kAhead && nt > 0) heads_of(0, &nb, &nc);
  for (int g = 0; g < groups; ++g) {
    float xv[kGroup], s[kGroup], y[kGroup], z[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      xv[k] = value_of<DT>(nx[k]);
      s[k] = value_of<DT>(ndt[k]) + bias;
      if (MODE == kScanOut) z[k] = value_of<DT>(nz[k]);
    }
    if (g + 1 < groups) fetch();
    if (a.softplus) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k) s[k] = softplus(s[k]);
    }
#pragma unroll
    for (int k = 0; k < kGroup; ++k) y[k] = token(xv[k], s[k], g * kGroup + k);
    if (MODE == kScanOut) {
      if (pz) {
#pragma unroll
        for (int k = 0; k < kGroup; ++k) y[k] *= z[k] * sigmoidf(z[k]);
      }
      if (mine) {
        const unsigned o = lane_offset(off);
#pragma unroll
        for (int k = 0; k < kGroup; ++k) Elem<DT>::store(reinterpret_cast<char*>(out + k * a.os[1]) + o, 0, y[k]);
      }
      out += kGroup * a.os[1];
    }
  }
  for (int t = groups * kGroup; t < nt; ++t) {     // fewer than a group
    const float xv = value_of<DT>(take(px, a.xs[1], off));
    float s = value_of<DT>(take(pdt, a.dts[1], off)) + bias;
    if (a.softplus) s = softplus(s);
    float y = token(xv, s, t);
    if (MODE == kScanOut) {
      if (pz) {
        const float z = value_of<DT>(take(pz, a.zs[1], off));
        y *= z * sigmoidf(z);
      }
      if (mine) Elem<DT>::store(reinterpret_cast<char*>(out) + off, 0, y);
      out += a.os[1];
    }
  }
  if (!mine) return;
  if (MODE == kScanState) {
    store_states<NS>(a.seg_state + (piece * a.D + d) * a.n, a.n, a.n % 4 == 0, h);
    a.seg_step[piece * a.D + d] = total;
    return;
  }
  if (p.piece == last && slot >= 0 && a.state_out) store_states<NS>(a.state_out + sb, a.n, a.n % 4 == 0, h);
  if (a.zero_rest) {
    const int64_t rows = min(p.own - first, static_cast<int64_t>(a.q.len));
    for (int64_t t = max(nt, 0); t < rows; ++t, out += a.os[1]) Elem<DT>::store(out, d, 0.f);
  }
}

// Four values, or one, of B or C: four in one load at any element's address.
template <int DT, int VEC>
struct Few {
  Raw<DT, 4, kOdd> r;
  __device__ __forceinline__ void load(const void* p, int64_t i) { r.load(p, i, 4); }
  __device__ __forceinline__ float value(int i) const { return r.value(i); }
};
template <int DT>
struct Few<DT, 1> {
  float v;
  __device__ __forceinline__ void load(const void* p, int64_t i) { v = Elem<DT>::load(p, i); }
  __device__ __forceinline__ float value(int) const { return v; }
};

// The state at the start of each segment of sequence blockIdx.y, from what the segments before it add,
// in place: a thread a state.
__global__ void __launch_bounds__(256) scan_carry(ScanArgs a) {
  const int s = blockIdx.y;
  Span p;
  seq_span(a.q, s, &p);
  const int pieces = p.len > 0 ? (p.len - 1) / a.q.len + 1 : 1;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, all = static_cast<int64_t>(a.D) * a.n;
  if (pieces < 2 || i >= all) return;
  const int64_t w0 = a.q.T > 0 ? p.row0 / a.q.len + s : static_cast<int64_t>(s) * a.q.n_seg;
  const int slot = seq_slot(a.slots, a.n_slots, s);
  const int d = static_cast<int>(i / a.n);
  const float A2 = in_log2(a.A[i]);
  float h = slot >= 0 && a.state_in ? a.state_in[slot * all + i] : 0.f;
  float* to = a.seg_state + w0 * all + i;
  const float* step = a.seg_step + w0 * a.D + d;
  constexpr int kAhead = 16;
  for (int g0 = 0; g0 < pieces; g0 += kAhead) {
    float own[kAhead], total[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const bool there = g0 + k < pieces - 1;       // (the last one adds nothing to a later one)
      own[k] = there ? to[(g0 + k) * all] : 0.f;
      total[k] = there ? step[static_cast<int64_t>(g0 + k) * a.D] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (g0 + k < pieces) to[(g0 + k) * all] = h;
      h = fmaf(__builtin_amdgcn_exp2f(total[k] * A2), h, own[k]);
    }
  }
}

// One token a sequence: P lanes (a power of two) share a channel's states, VEC each, and a thread takes
// the same states of U sequences, whose loads it asks for at once.
template <int DT, int VEC, int U>
__global__ void __launch_bounds__(256) scan_step(ScanArgs a, int P) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t d = at / P;
  const int n0 = static_cast<int>(at - d * P) * VEC;
  if (d >= a.D) return;                             // (whole channels: P divides 64)
  const bool some = n0 < a.n;
  typedef float vec __attribute__((ext_vector_type(VEC)));
  const int64_t g = d / (a.D / a.G);
  int slot[U];
  vec h[U];
  Few<DT, VEC> b[U], c[U];
  float x[U], step[U], z[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int s = blockIdx.y * U + u;
    slot[u] = s < a.q.S ? seq_slot(a.slots, a.n_slots, s) : -1;
    if (slot[u] >= 0) {
      if (some) {
        h[u] = __builtin_nontemporal_load(reinterpret_cast<const vec*>(a.state_in + (static_cast<int64_t>(slot[u]) * a.D + d) * a.n + n0));
        b[u].load(a.b, s * a.bs[0] + g * a.bs[1] + n0);
        c[u].load(a.c, s * a.cs[0] + g * a.cs[1] + n0);
      }
      x[u] = Elem<DT>::load(a.x, s * a.xs[0] + d);
      step[u] = Elem<DT>::load(a.dt, s * a.dts[0] + d);
      z[u] = a.z ? Elem<DT>::load(a.z, s * a.zs[0] + d) : 0.f;
    }
  }
  vec A = {};
  if (some) A = *reinterpret_cast<const vec*>(a.A + d * a.n + n0);
  const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int s = blockIdx.y * U + u;
    if (s >= a.q.S) return;
    if (slot[u] < 0) {
      if (n0 == 0) Elem<DT>::store(a.out, s * a.os[0] + d, 0.f);
      continue;
    }
    float D = step[u] + bias, y = 0.f;
    if (a.softplus) D = softplus(D);
    if (some) {
      vec to;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        to[i] = fmaf(__builtin_amdgcn_exp2f(D * in_log2(A[i])), h[u][i], D * x[u] * b[u].value(i));
        y = fmaf(c[u].value(i), to[i], y);
      }
      __builtin_nontemporal_store(to, reinterpret_cast<vec*>(a.state_out + (static_cast<int64_t>(slot[u]) * a.D + d) * a.n + n0));
    }
    for (int o = 1; o < P; o *= 2) y += __shfl_xor(y, o);
    if (n0 == 0) {
      y = fmaf(skip, x[u], y);
      if (a.z) y *= z[u] * sigmoidf(z[u]);
      Elem<DT>::store(a.out, s * a.os[0] + d, y);
    }
  }
}

template <int DT, int NS, bool FAST>
hipError_t launch_rows(const ScanArgs& a, bool state, hipStream_t st) {
  const int64_t x = static_cast<int64_t>(a.tiles) * a.G;
  const int waves = static_cast<int>(std::min<int64_t>(x, 4));
  const dim3 grid = seq_grid(a.q, (x + waves - 1) / waves), block(64 * waves);
  if (state) hipLaunchKernelGGL((scan_rows<DT, NS, FAST, kScanState>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((scan_rows<DT, NS, FAST, kScanOut>), grid, block, 0, st, a);
  return hipGetLastError();
}
template <int DT, int NS>
hipError_t launch_how(const ScanArgs& a, bool state, hipStream_t st) {
  return scan_fast(a, DT, NS) ? launch_rows<DT, NS, true>(a, state, st) : launch_rows<DT, NS, false>(a, state, st);
}
template <int DT>
hipError_t launch_n(const ScanArgs& a, bool state, hipStream_t st) {
  if (a.n <= 4) return launch_how<DT, 4>(a, state, st);
  if (a.n <= 8) return launch_how<DT, 8>(a, state, st);
  if (a.n <= 12) return launch_how<DT, 12>(a, state, st);
  if (a.n <= 16) return launch_how<DT, 16>(a, state, st);
  if (a.n <= 24) return launch_how<DT, 24>(a, state, st);
  if (a.n <= 32) return launch_how<DT, 32>(a, state, st);
  if (a.n <= 48) return launch_how<DT, 48>(a, state, st);
  return launch_how<DT, 64>(a, state, st);
}
hipError_t launch_pass(const ScanArgs& a, int dt, bool state, hipStream_t st) {
  return dt == RN_F32 ? launch_n<RN_F32>(a, state, st) : launch_n<RN_BF16>(a, state, st);
}

template <int DT, int VEC>
hipError_t launch_step(const ScanArgs& a, int P, hipStream_t st) {
  const int64_t x = (static_cast<int64_t>(a.D) * P + 255) / 256;
  // Two sequences a thread where that leaves the chip eight blocks a CU and more: A is read once for them. (128
  // sequences of 4096 channels x 16 states, bf16, 24 such pools in turn: 18.1 us, of which the states' 67 MB
  // take 14 at a large copy's rate; four a thread 19.1; through the caches 20.9. Two pools in turn, which the
  // last-level cache holds: 17.6 and through the caches 16.2.)
  if (x * a.q.S >= 4096) {
    hipLaunchKernelGGL((scan_step<DT, VEC, 2>), dim3(static_cast<unsigned>(x), (a.q.S + 1) / 2), dim3(256), 0, st, a, P);
  } else {
    hipLaunchKernelGGL((scan_step<DT, VEC, 1>), dim3(static_cast<unsigned>(x), a.q.S), dim3(256), 0, st, a, P);
  }
  return hipGetLastError();
}

// Tokens a segment. Whole sequences where their channels make a wave or more for each of the chip's 1024
// SIMDs (bf16 with gate, 16 states, 4096 channels: 32 sequences of 512 tokens 295 us, cut 442; 24: 292 and
// 343; 16: 231 and 227; 12 of 1024: 470 and 323), or where the sequences are short (8 of 32 tokens, 1000
// channels, 12 states, float32: 20 and 28 us; of 64: 28 and 28); sequences of unknown lengths count as so many
// of the longest's. Else 10 waves a SIMD in all: about 5 are there at once, and more take turns better than one
// round of waves, half as many again being slower for the states that pass between them (8192 tokens of
// 4096 channels: 232 us; 4 to 7 waves: 246 to 261, 12: 234).
int segment(const ScanCall& c) {
  const int64_t per = static_cast<int64_t>(c.G) * ((c.D / c.G + 63) / 64);
  const int64_t tokens = c.T > 0 ? std::min<int64_t>(c.T, static_cast<int64_t>(c.S) * c.N) : static_cast<int64_t>(c.S) * c.N;
  const int64_t L = std::max<int64_t>((tokens * per / 10240 + 15) / 16 * 16, 16);
  if (c.N < 64 || 2 * L > c.N || tokens * per >= 1280 * static_cast<int64_t>(c.N)) return c.N;
  return static_cast<int>(L);
}

}  // namespace

size_t scan_ws_bytes(const ScanCall& c) {
  const ScanArgs a = scan_args(c, segment(c));
  if (a.q.n_seg < 2) return 0;
  const size_t rows = static_cast<size_t>(seq_pieces(a.q));
  return rows * c.D * c.n * sizeof(float) + rows * c.D * sizeof(float);
}

hipError_t launch_selective_scan(const ScanCall& c, hipStream_t st) {
  ScanArgs a = scan_args(c, segment(c));
  if (a.q.n_seg < 2) return launch_pass(a, c.type, false, st);
  const size_t rows = static_cast<size_t>(seq_pieces(a.q));
  a.seg_state = static_cast<float*>(c.ws);
  a.seg_step = a.seg_state + rows * c.D * c.n;
  hipError_t e = launch_pass(a, c.type, true, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(scan_carry, dim3(static_cast<unsigned>((static_cast<int64_t>(c.D) * c.n + 255) / 256), c.S), dim3(256), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return launch_pass(a, c.type, false, st);
}

hipError_t launch_selective_step(const ScanCall& c, hipStream_t st) {
  const ScanArgs a = scan_args(c, 1);
  const int vec = c.n % 4 == 0 && reinterpret_cast<uintptr_t>(c.A) % 16 == 0 ? 4 : 1;
  int P = 1;
  while (P * vec < c.n) P *= 2;
  if (c.type == RN_F32) return vec == 4 ? launch_step<RN_F32, 4>(a, P, st) : launch_step<RN_F32, 1>(a, P, st);
  return vec == 4 ? launch_step<RN_BF16, 4>(a, P, st) : launch_step<RN_BF16, 1>(a, P, st);
}

}  // namespace rn
