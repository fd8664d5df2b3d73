// Selective scan: prompts (selective_scan.h) and single tokens.
//
// Prompts. Bound by the vector units: for 16 states, a channel and token take 16 (5 instructions, one of
// them an exponential at half the rate) and about 40 more. A sequence whose channels do not fill the chip
// is cut into segments: one pass gives the state that each adds on its own, scan_carry carries the states
// over the segments, a second pass gives the outputs.
//
// Single tokens. Bound by HBM: the float32 state is read and written once.
#include <algorithm>

#include "selective_scan.h"

namespace rn {
namespace {

// Where a kernel starts and ends: a whole sequence, or a segment whose starting state is in the
// workspace; or the state a segment adds on its own.
enum ScanMode : int { kScanOut = 0, kScanState = 1 };

template <int DT, int NS, bool FAST, ScanMode MODE>
__global__ void __launch_bounds__(256) scan_rows(ScanArgs a) {
  __shared__ float2 steps[kTile][64];     // D_t and D_t x_t
  __shared__ float parts[MODE == kScanOut ? 4 : 1][kTile][64];
  Span p;
  const int64_t piece = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
  if (!seq_place(a.q, piece, &p)) return;
  const int len = __builtin_amdgcn_readfirstlane(p.len);
  p.piece = __builtin_amdgcn_readfirstlane(p.piece);
  const int first = p.piece * a.q.len;
  const int last = len > 0 ? (len - 1) / a.q.len : 0;      // the piece that ends the sequence
  if (MODE == kScanState && p.piece >= last) return;
  const int nt = min(len - first, a.q.len);                // tokens of the piece
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = blockIdx.x / a.tiles, each = a.D / a.G;
  const int in_group = (blockIdx.x - group * a.tiles) * 64 + lane;
  const bool mine = in_group < each;
  const int d = group * each + in_group;
  const int n0 = wave * NS, have = min(NS, a.n - n0);      // this wave's states (have <= 0: none)
  const int waves = (a.n + NS - 1) / NS;
  const int64_t row0 = uniform64(p.row0);
  auto base = [&](const int64_t* st) {
    return (a.q.T > 0 ? row0 * st[1] : p.s * st[0]) + static_cast<int64_t>(first) * st[1];
  };
  const int64_t xb = base(a.xs) + d, dtb = base(a.dts) + d, zb = base(a.zs) + d, ob = base(a.os) + d;
  auto base3 = [&](const int64_t* st) {
    return (a.q.T > 0 ? row0 * st[2] : p.s * st[0]) + group * st[1] + static_cast<int64_t>(first) * st[2] + n0;
  };
  const int64_t bb = base3(a.bs), cb = base3(a.cs);
  float A2[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] = mine && i < have ? a.A[static_cast<int64_t>(d) * a.n + n0 + i] * kLog2e : 0.f;
    h[i] = 0.f;
  }
  const float skip = mine && a.skip ? a.skip[d] : 0.f, bias = mine && a.bias ? a.bias[d] : 0.f;
  const int slot = p.s < a.q.S ? seq_slot(a.slots, a.n_slots, p.s) : -1;
  const int64_t sb = (static_cast<int64_t>(slot) * a.D + d) * a.n + n0;
  if (MODE == kScanOut && mine) {
    const float* from = p.piece <= last && last > 0 ? a.seg_state + (piece * a.D + d) * a.n + n0
                        : slot >= 0 && a.state_in && p.piece == 0 ? a.state_in + sb : nullptr;
    if (from) {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < have) h[i] = from[i];
    }
  }
  float total = 0.f;                      // kScanState: the sum of D_t
  float nx[kEach], ndt[kEach], nz[kEach];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int t = t0 + wave * kEach + k;
      const bool there = mine && t < nt;
      nx[k] = there ? Elem<DT>::load(a.x, xb + t * a.xs[1]) : 0.f;
      ndt[k] = there ? Elem<DT>::load(a.dt, dtb + t * a.dts[1]) : 0.f;
      if (MODE == kScanOut) nz[k] = there && a.z ? Elem<DT>::load(a.z, zb + t * a.zs[1]) : 0.f;
    }
  };
  fetch(0);
  for (int t0 = 0; t0 < nt; t0 += kTile) {
    float x[kEach], z[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int t = wave * kEach + k;
      float s = ndt[k] + bias;
      if (a.softplus) s = softplus(s);
      if (t0 + t >= nt) s = 0.f;
      steps[t][lane] = make_float2(s, s * nx[k]);
      x[k] = nx[k];
      z[k] = nz[k];
    }
    if (t0 + kTile < nt) fetch(t0 + kTile);
    __syncthreads();
    if (have > 0) {
      auto token = [&](int t, const Uniform<DT, NS, FAST>& b, const Uniform<DT, NS, FAST>& c) {
        const float2 s = steps[t][lane];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          h[i] = fmaf(__builtin_amdgcn_exp2f(s.x * A2[i]), h[i], s.y * b.value(i));
          if (MODE == kScanOut) y = fmaf(c.value(i), h[i], y);
        }
        if (MODE == kScanOut) parts[wave][t][lane] = y;
        else total += s.x;
      };
      if (t0 + kTile <= nt) {
#pragma unroll 4
        for (int t = 0; t < kTile; ++t) {
          Uniform<DT, NS, FAST> b, c;
          b.load(a.b, bb + (t0 + t) * a.bs[2], have);
          if (MODE == kScanOut) c.load(a.c, cb + (t0 + t) * a.cs[2], have);
          token(t, b, c);
        }
      } else {
        for (int t = 0; t < nt - t0; ++t) {
          Uniform<DT, NS, FAST> b, c;
          b.load(a.b, bb + (t0 + t) * a.bs[2], have);
          if (MODE == kScanOut) c.load(a.c, cb + (t0 + t) * a.cs[2], have);
          token(t, b, c);
        }
      }
    }
    __syncthreads();
    if (MODE == kScanOut) {
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int t = wave * kEach + k;
        if (mine && t0 + t < nt) {
          float y = skip * x[k];
          for (int w = 0; w < waves; ++w) y += parts[w][t][lane];
          if (a.z) y *= z[k] * sigmoidf(z[k]);
          Elem<DT>::store(a.out, ob + (t0 + t) * a.os[1], y);
        }
      }
    }
  }
  if (MODE == kScanState) {
    if (mine) {
      float* to = a.seg_state + (piece * a.D + d) * a.n + n0;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < have) to[i] = h[i];
      if (wave == 0) a.seg_step[piece * a.D + d] = total;
    }
    return;
  }
  if (mine && p.piece == last && slot >= 0 && a.state_out) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (i < have) a.state_out[sb + i] = h[i];
  }
  if (a.zero_rest && mine) {
    const int64_t rows = min(p.own - first, static_cast<int64_t>(a.q.len));
    for (int64_t t = max(nt, 0) + wave; t < rows; t += 4) Elem<DT>::store(a.out, ob + t * a.os[1], 0.f);
  }
}

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
  const float A2 = a.A[i] * kLog2e;
  float h = slot >= 0 && a.state_in ? a.state_in[slot * all + i] : 0.f;
  float* to = a.seg_state + w0 * all + i;
  const float* step = a.seg_step + w0 * a.D + d;
  constexpr int kAhead = 8;
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

// One token a sequence: P lanes (a power of two) share a channel's states, VEC each.
template <int DT, int VEC>
__global__ void __launch_bounds__(256) scan_step(ScanArgs a, int P) {
  const int s = blockIdx.y;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t d = at / P;
  const int n0 = static_cast<int>(at - d * P) * VEC;
  if (d >= a.D) return;                             // (whole channels: P divides 64)
  const bool some = n0 < a.n;
  const int slot = seq_slot(a.slots, a.n_slots, s);
  const int64_t ob = s * a.os[0] + d;
  if (slot < 0) {
    if (n0 == 0) Elem<DT>::store(a.out, ob, 0.f);
    return;
  }
  typedef float vec __attribute__((ext_vector_type(VEC)));
  float h[VEC], A[VEC], b[VEC], c[VEC];
  const int64_t sb = (static_cast<int64_t>(slot) * a.D + d) * a.n + n0;
  const int64_t g = d / (a.D / a.G);
#pragma unroll
  for (int i = 0; i < VEC; ++i) h[i] = A[i] = b[i] = c[i] = 0.f;
  if (some) {
    const vec hv = __builtin_nontemporal_load(reinterpret_cast<const vec*>(a.state_in + sb));
    const vec Av = *reinterpret_cast<const vec*>(a.A + d * a.n + n0);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      h[i] = hv[i];
      A[i] = Av[i];
      b[i] = Elem<DT>::load(a.b, s * a.bs[0] + g * a.bs[1] + n0 + i);
      c[i] = Elem<DT>::load(a.c, s * a.cs[0] + g * a.cs[1] + n0 + i);
    }
  }
  const float x = Elem<DT>::load(a.x, s * a.xs[0] + d);
  float step = Elem<DT>::load(a.dt, s * a.dts[0] + d) + (a.bias ? a.bias[d] : 0.f);
  if (a.softplus) step = softplus(step);
  float y = 0.f;
  vec to;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    h[i] = fmaf(__builtin_amdgcn_exp2f(step * (A[i] * kLog2e)), h[i], step * x * b[i]);
    y = fmaf(c[i], h[i], y);
    to[i] = h[i];
  }
  if (some) __builtin_nontemporal_store(to, reinterpret_cast<vec*>(a.state_out + sb));
  for (int o = 1; o < P; o *= 2) y += __shfl_xor(y, o);
  if (n0 == 0) {
    if (a.skip) y = fmaf(a.skip[d], x, y);
    if (a.z) {
      const float z = Elem<DT>::load(a.z, s * a.zs[0] + d);
      y *= z * sigmoidf(z);
    }
    Elem<DT>::store(a.out, ob, y);
  }
}

template <int DT, int NS, bool FAST>
hipError_t launch_rows(const ScanArgs& a, bool state, hipStream_t st) {
  const dim3 grid = seq_grid(a.q, static_cast<int64_t>(a.tiles) * a.G);
  if (state) hipLaunchKernelGGL((scan_rows<DT, NS, FAST, kScanState>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((scan_rows<DT, NS, FAST, kScanOut>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}
template <int DT, bool FAST>
hipError_t launch_n(const ScanArgs& a, bool state, hipStream_t st) {
  switch (scan_states(a.n)) {
    case 2: return launch_rows<DT, 2, FAST>(a, state, st);
    case 4: return launch_rows<DT, 4, FAST>(a, state, st);
    case 8: return launch_rows<DT, 8, FAST>(a, state, st);
    default: return launch_rows<DT, 16, FAST>(a, state, st);
  }
}
hipError_t launch_pass(const ScanArgs& a, int dt, bool state, hipStream_t st) {
  const bool fast = scan_fast(a, dt);
  if (dt == RN_F32) return fast ? launch_n<RN_F32, true>(a, state, st) : launch_n<RN_F32, false>(a, state, st);
  return fast ? launch_n<RN_BF16, true>(a, state, st) : launch_n<RN_BF16, false>(a, state, st);
}

// Tokens a segment: whole sequences where their channels fill the chip by themselves (three blocks of
// four waves a CU); else as many segments as do.
int segment(const ScanCall& c) {
  const int64_t per = static_cast<int64_t>(c.G) * ((c.D / c.G + 63) / 64);
  const int64_t tokens = c.T > 0 ? std::min<int64_t>(c.T, static_cast<int64_t>(c.S) * c.N) : static_cast<int64_t>(c.S) * c.N;
  int64_t L = std::max<int64_t>((tokens * per / 1024 + 15) / 16 * 16, 64);
  if (2 * L > c.N) L = c.N;
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
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(c.D) * P + 255) / 256), c.S);
  if (c.type == RN_F32) {
    if (vec == 4) hipLaunchKernelGGL((scan_step<RN_F32, 4>), grid, dim3(256), 0, st, a, P);
    else hipLaunchKernelGGL((scan_step<RN_F32, 1>), grid, dim3(256), 0, st, a, P);
  } else {
    if (vec == 4) hipLaunchKernelGGL((scan_step<RN_BF16, 4>), grid, dim3(256), 0, st, a, P);
    else hipLaunchKernelGGL((scan_step<RN_BF16, 1>), grid, dim3(256), 0, st, a, P);
  }
  return hipGetLastError();
}

}  // namespace rn
